"""CPU: sizes at the ends of what the plans of the rotation, the state cache and the context operators hold."""
import math
import os

import numpy as np
import pytest


def _sn():
    import schnet_cfconv_force_amd as sn
    if not os.path.exists(sn.LIB_PATH):
        from schnet_cfconv_force_amd import build
        build.build(verbose=False)
    return sn


# ------------------------------------------------------------------ numbers beyond 32 bits

@pytest.mark.parametrize("over", [2 ** 31, 2 ** 32, -2 ** 31 - 100, -2 ** 32])
def test_plans_refuse_sizes_that_32_bits_do_not_hold(over):
    """The lowest 32 bits of each would be a size that the plan takes."""
    sn = _sn()
    cache = sn.StateCache(4, 16, 2, 32, device="cpu")
    for size, good in (("window", 5), ("max_pages", 4), ("n_heads", 4)):
        with pytest.raises(ValueError):
            sn.CacheRows(cache, [0, 1], **{"max_pages": 4, size: good + over})
    for size, good in (("n_pages", 4), ("page_size", 16), ("n_kv_heads", 2), ("head_dim", 32)):
        with pytest.raises(ValueError):
            sn.StateCache(**{"n_pages": 4, "page_size": 16, "n_kv_heads": 2, "head_dim": 32, size: good + over}, device="cpu")
    for size, good in (("n_rows", 5), ("n_heads", 4), ("head_dim", 32), ("n_kv_heads", 2)):
        with pytest.raises(ValueError):
            sn.HeadRotary(**{"n_rows": 5, "n_heads": 4, "head_dim": 32, size: good + over}, device="cpu")
    with pytest.raises(ValueError):
        sn.HeadRotary(5, 4, 32, freqs=[1.0, 2.0], axes=np.array([0, 1 + over]), device="cpu")
    with pytest.raises(ValueError):
        sn.rotary_frequencies(np.array([4, 4 + over]))
    for size, good in (("n_heads", 4), ("n_kv_heads", 2), ("head_dim", 32)):
        with pytest.raises(ValueError):
            sn.CrossAttention([0, 1], [0, 1], **{"n_heads": 4, "n_kv_heads": 2, "head_dim": 32, size: good + over}, device="cpu")
    with pytest.raises(ValueError):
        sn.CrossAttention([0, 1], [0, 1], 4, 2, 32, thresholds=np.array([-1, 0, 1 + over]), device="cpu")
    for size, good in (("n_channels", 32), ("n_groups", 4)):
        with pytest.raises(ValueError):
            sn.GroupNorm([0, 1], **{"n_channels": 32, "n_groups": 4, size: good + over}, device="cpu")


def test_windows_and_scales_at_the_ends_of_32_bits():
    sn = _sn()
    cache = sn.StateCache(4, 16, 2, 32, device="cpu")
    plan = sn.CacheRows(cache, [0, 1], 4, window=2 ** 31 - 1, scale=float(np.finfo(np.float32).max))
    assert plan.c.window == 2 ** 31 - 1 and math.isfinite(plan.c.scale)
    for scale in (1e39, -1e39, math.nan):
        with pytest.raises(ValueError):
            sn.CacheRows(cache, [0, 1], 4, scale=scale)

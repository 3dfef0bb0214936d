"""CPU: sizes at the ends of what the plans of the rotation, the state cache and the context operators hold."""
import ctypes
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


# ------------------------------------------------------------------ many rows

def test_plans_of_more_rows_than_an_attention_holds_write_and_read():
    """Their workspace is the status words alone, and an attention is refused before any GPU work."""
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnCache

    def desc(B, n_rows, max_rows, max_pages, n_heads=4):
        return S(9, 1024, 2, 32, sn.SN_BF16, sn.SN_CODES_INT8, 256, 256, 256, 256, B, n_rows, max_rows, max_pages, 256, 256, 256, n_heads,
                 0.5, 1, 0, 256, 128, 32)

    for d in (desc(32, 32 * 65536, 65536, 64, 64), desc(256, 65536 + 255, 65536, 64, 512), desc(65535, 65536, 65536, 64),
              desc(1, 2 ** 29, 2 ** 29, 2 ** 19), desc(1, 2 ** 28, 2 ** 28, 2 ** 18, 8)):
        assert lib.sn_cache_workspace_bytes(ctypes.byref(d)) == 256
        assert lib.sn_cache_attend(ctypes.byref(d), 256, None, 256, 1 << 40, None) == sn.SN_ERR_INVALID
        # past the sizes, to the rows' addresses
        assert lib.sn_cache_write(ctypes.byref(d), None, 64, 32, 256, 64, 32, 256, 256, None) == sn.SN_ERR_INVALID
        assert lib.sn_cache_read(ctypes.byref(d), None, 256, 256, 255, None) == sn.SN_ERR_WORKSPACE
    # the largest that an attention's launch holds, and the next
    assert lib.sn_cache_workspace_bytes(ctypes.byref(desc(2, 8 * 2 ** 18, 8 * 2 ** 18 - 16, 2 ** 11))) > 256
    for B, max_rows, held in ((1, 2 ** 25 - 40, True), (1, 2 ** 25 - 24, False)):
        d = desc(B, max_rows, max_rows, 2 ** 15)
        assert (lib.sn_cache_workspace_bytes(ctypes.byref(d)) > 256) == held
    cache = sn.StateCache(4, 1024, 2, 32, device="cpu")
    plan = sn.CacheRows(cache, np.concatenate([[0], np.full(256, 65536)]).cumsum()[:33], 64, n_heads=64)
    assert plan.workspace_bytes == 256


# ------------------------------------------------------------------ frequencies

def test_frequencies_whose_angles_fp64_does_not_hold_are_refused():
    """A position times the largest finite numbers is infinite, and its sine not a number."""
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnHeadRotary
    axes = np.zeros(1, np.int32)
    for freq, fine in ((1e308, False), (-1e308, False), (2.0 ** 52, False), (2.0 ** 51, True)):
        freqs = np.array([freq])
        d = S(6, 4, 2, 32, sn.SN_BF16, 0, 1e-6, 1, 1, 0, freqs.ctypes.data, axes.ctypes.data, 256, 256, 256, 128, 32, 64, 32, None, None)
        # behind the descriptor comes the workspace
        assert lib.sn_head_rotary_forward(ctypes.byref(d), None, 256, 256, 0, None) == (sn.SN_ERR_WORKSPACE if fine else sn.SN_ERR_INVALID)
        if fine:
            sn.HeadRotary(6, 4, 32, freqs=freqs, device="cpu")
        else:
            with pytest.raises(ValueError):
                sn.HeadRotary(6, 4, 32, freqs=freqs, device="cpu")
    for base in (5e-324, 1e-300, 1e-20):
        with pytest.raises(sn.SnError):
            sn.rotary_frequencies([40], base)
    assert np.allclose(sn.rotary_frequencies([4], 2.0 ** -8)[0], [1, 4, 16, 64])

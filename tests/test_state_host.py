"""CPU checks of the rotation of heads and of the state cache: what the plans, the calls and the C entry points refuse
before any GPU work, the frequencies, and the 64-bit references against central differences."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import state_ref as R


def _sn():
    import schnet_cfconv_force_amd as sn
    if not os.path.exists(sn.LIB_PATH):
        from schnet_cfconv_force_amd import build
        build.build(verbose=False)
    return sn


# ------------------------------------------------------------------ frequencies

def test_frequencies_fall_by_the_ladder():
    sn = _sn()
    freqs, axes = sn.rotary_frequencies([16, 24, 24])
    assert freqs.dtype == np.float64 and axes.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    assert np.allclose(freqs, 10000.0 ** (-np.arange(64) / 64), rtol=1e-14)
    freqs, axes = sn.rotary_frequencies([2, 3], base=100.0, shared=False)
    assert np.allclose(freqs, [1, 0.1, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-14) and axes.tolist() == [0, 0, 1, 1, 1]


@pytest.mark.parametrize("sections,base", [([], 1e4), ([0], 1e4), ([3, -1], 1e4), ([65], 1e4), ([60, 5], 1e4), ([1] * 9, 1e4),
                                           ([4], 0.0), ([4], -2.0), ([4], math.inf), ([4], math.nan), ([2 ** 30] * 3, 1e4)])
def test_frequencies_refuse(sections, base):
    sn = _sn()
    with pytest.raises(sn.SnError) as e:
        sn.rotary_frequencies(sections, base)
    assert e.value.status == sn.SN_ERR_INVALID


# ------------------------------------------------------------------ plans and tensors

def test_rotary_plans_refuse():
    sn = _sn()
    make = lambda *a, **k: sn.HeadRotary(*a, device="cpu", **k)  # noqa: E731
    for change in ({"n_rows": -1}, {"n_heads": 0}, {"head_dim": 0}, {"head_dim": 129}, {"n_kv_heads": -1}, {"n_heads": 70000},
                   {"freqs": [1.0] * 17}, {"freqs": [1.0], "axes": [8]}, {"n_rows": 2 ** 31 - 1}):
        args = {"n_rows": 5, "n_heads": 4, "head_dim": 32, **change}
        with pytest.raises(sn.SnError):
            make(**args)
    for change in ({"freqs": [1.0], "axes": [-1]}, {"freqs": [math.nan]}, {"freqs": [1.0, 2.0], "axes": [0]}, {"eps": 0.0}, {"eps": 1e-40},
                   {"eps": math.inf}, {"dtype": torch.float16}):
        with pytest.raises(ValueError):
            make(5, 4, 32, **change)


def test_rotary_calls_refuse_tensors_that_do_not_fit():
    sn = _sn()
    plan = sn.HeadRotary(3, 4, 32, n_kv_heads=2, freqs=[1.0, 0.1], axes=[0, 1], device="cpu")
    good = {"q": torch.zeros(3, 4, 32), "k": torch.zeros(3, 2, 32), "positions": torch.zeros(2, 3, dtype=torch.int32),
            "q_weight": None, "k_weight": None}
    plan._bind(**good)
    for change in ({"q": torch.zeros(3, 4, 31)}, {"q": torch.zeros(2, 4, 32)}, {"q": torch.zeros(3, 4, 32).bfloat16()},
                   {"k": None}, {"k": torch.zeros(3, 4, 32)}, {"k": torch.zeros(3, 2, 64)[:, :, ::2]}, {"positions": None},
                   {"positions": torch.zeros(3, 2, dtype=torch.int32)}, {"positions": torch.zeros(2, 3)},
                   {"positions": torch.zeros(2, 6, dtype=torch.int32)[:, ::2]}, {"q_weight": torch.ones(31)},
                   {"k_weight": torch.ones(32).double()}):
        with pytest.raises(ValueError):
            plan._bind(**{**good, **change})
    with pytest.raises(ValueError):     # a weight without a norm
        sn.HeadRotary(3, 4, 32, n_kv_heads=2, norm=False, device="cpu")._bind(**{**good, "positions": None, "q_weight": torch.ones(32)})
    with pytest.raises(ValueError):     # keys without key heads
        sn.HeadRotary(3, 4, 32, device="cpu")._bind(**{**good, "positions": None})


def test_cache_plans_refuse():
    sn = _sn()
    make = lambda *a, **k: sn.StateCache(*a, device="cpu", **k)  # noqa: E731
    for args in ((0, 16, 2, 32), (4, 8, 2, 32), (4, 24, 2, 32), (4, 2048, 2, 32), (4, 16, 0, 32), (4, 16, 2, 0), (4, 16, 2, 129)):
        with pytest.raises(sn.SnError):
            make(*args)
    with pytest.raises(ValueError):
        make(4, 16, 2, 32, dtype=torch.float16)
    with pytest.raises(ValueError):
        make(4, 16, 2, 32, codes="int4")
    cache = make(4, 16, 2, 40, codes="e4m3")
    assert cache.k.shape == (4, 2, 16, 40) and cache.k.stride() == (2 * 16 * 48, 16 * 48, 48, 1)
    for row_ptr in ([0], [1, 2], [0, 3, 2], [0, 2 ** 31]):
        with pytest.raises(ValueError):
            sn.CacheRows(cache, row_ptr, 4)
    with pytest.raises(ValueError):
        sn.CacheRows(cache, [0, 1], 4, scale=math.inf)
    for change in ({"max_pages": 0}, {"max_pages": 2 ** 28}, {"n_heads": 3}, {"n_heads": 0}, {"window": -1},
                   {"window": 4, "causal": False}):
        with pytest.raises(sn.SnError):
            sn.CacheRows(cache, [0, 1], **{"max_pages": 4, **change})


def test_cache_calls_refuse_tensors_that_do_not_fit():
    sn = _sn()
    cache = sn.StateCache(4, 16, 2, 32, device="cpu")
    plan = sn.CacheRows(cache, [0, 1, 3], 5, n_heads=4)
    good = {"table": torch.zeros(2, 5, dtype=torch.int32), "lengths": torch.zeros(2, dtype=torch.int32), "q": torch.zeros(3, 4, 32)}
    plan._bind(**good)
    for change in ({"table": None}, {"lengths": None}, {"table": torch.zeros(2, 4, dtype=torch.int32)}, {"table": torch.zeros(2, 5)},
                   {"table": torch.zeros(2, 10, dtype=torch.int32)[:, ::2]}, {"lengths": torch.zeros(2, dtype=torch.int64)},
                   {"lengths": torch.zeros(3, dtype=torch.int32)}, {"q": torch.zeros(3, 2, 32)}, {"q": torch.zeros(3, 4, 32).bfloat16()}):
        with pytest.raises(ValueError):
            plan._bind(**{**good, **change})


def test_calls_refuse_a_workspace_on_the_host():
    """Before the library is reached: the kernels would write there."""
    sn = _sn()
    cache = sn.StateCache(4, 16, 2, 32, device="cpu")
    plan = sn.CacheRows(cache, [0, 1], 4)
    table, lengths = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    ws, rows = torch.zeros(1 << 12, dtype=torch.uint8), torch.zeros(1, 2, 32)
    rotary = sn.HeadRotary(1, 2, 32, n_kv_heads=2, device="cpu")
    for call in (lambda: sn.cache_write(plan, rows, rows, table, lengths, ws), lambda: sn.cache_read(plan, table, lengths, ws),
                 lambda: sn.cache_attend(plan, rows, table, lengths, ws),
                 lambda: sn.head_rotary_forward(rotary, rows, rows, None, ws),
                 lambda: sn.head_rotary_backward(rotary, rows, rows, None, rows, rows, ws)):
        with pytest.raises(ValueError, match="ws must be"):
            call()


# ------------------------------------------------------------------ the C entry points

def test_rotary_entry_points_refuse_before_any_gpu_work():
    """Dummy addresses that a GPU call would fault on: every check runs on the host."""
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnHeadRotary
    freqs, axes = np.ones(4), np.array([0, 1, 1, 0], np.int32)

    def desc(**change):
        d = S(6, 4, 2, 32, sn.SN_BF16, 1, 1e-6, 4, 2, 0, freqs.ctypes.data, axes.ctypes.data, 256, 256, 256, 128, 32, 64, 32, 256, 256)
        for name, value in change.items():
            setattr(d, name, value)
        return d

    def forward(d, q=256, k=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_head_rotary_forward(None if d is None else ctypes.byref(d), q, k, ws, ws_bytes, None)

    def backward(d, d_q=256, d_k=256, dq=256, dk=256, dqw=256, dkw=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_head_rotary_backward(None if d is None else ctypes.byref(d), d_q, 128, 32, d_k, 64, 32, dq, dk, dqw, dkw, ws,
                                           ws_bytes, None)

    assert forward(None) == sn.SN_ERR_INVALID and backward(None) == sn.SN_ERR_INVALID
    for change in ({"n_rows": -1}, {"n_heads": 0}, {"n_heads": 65536}, {"n_kv_heads": -1}, {"n_kv_heads": 65536}, {"head_dim": 0},
                   {"head_dim": 129}, {"dtype": 2}, {"norm": 2}, {"interleaved": -1}, {"n_pairs": -1}, {"n_pairs": 17}, {"n_axes": 0},
                   {"n_axes": 9}, {"n_rows": 2 ** 31 - 1}):
        d = desc(**change)
        assert lib.sn_head_rotary_workspace_bytes(ctypes.byref(d)) == 0, change
        assert forward(d) == sn.SN_ERR_INVALID and backward(d) == sn.SN_ERR_INVALID, change
    beyond, below, odd = np.array([0, 2, 1, 0], np.int32), np.array([0, -1, 1, 0], np.int32), np.array([1, math.inf, 1, 1.0])
    for change in ({"eps": 0.0}, {"eps": 1e-40}, {"eps": math.nan}, {"norm": 0}, {"freqs": None}, {"axes": None}, {"positions": None}, {"positions": 258},
                   {"q": None}, {"k": None}, {"q": 257}, {"k": 257}, {"q_weight": 258}, {"k_weight": 257}, {"axes": beyond.ctypes.data},
                   {"axes": below.ctypes.data}, {"freqs": odd.ctypes.data}):
        assert forward(desc(**change)) == sn.SN_ERR_INVALID and backward(desc(**change)) == sn.SN_ERR_INVALID, change
    d = desc()
    need = lib.sn_head_rotary_workspace_bytes(ctypes.byref(d))
    for ws, size in ((None, 1 << 40), (128, 1 << 40), (256, need - 1)):
        assert forward(d, ws=ws, ws_bytes=size) == sn.SN_ERR_WORKSPACE and backward(d, ws=ws, ws_bytes=size) == sn.SN_ERR_WORKSPACE
    for name in ("q", "k"):
        assert forward(d, **{name: None}) == sn.SN_ERR_INVALID and forward(d, **{name: 257}) == sn.SN_ERR_INVALID
    for name in ("d_q", "d_k", "dq", "dk"):
        assert backward(d, **{name: None}) == sn.SN_ERR_INVALID and backward(d, **{name: 257}) == sn.SN_ERR_INVALID
    assert backward(d, dqw=258) == sn.SN_ERR_INVALID
    assert backward(desc(norm=0, q_weight=None, k_weight=None)) == sn.SN_ERR_INVALID      # weights' gradients without a norm
    assert forward(desc(n_rows=0), q=None, k=None) == sn.SN_OK


def test_cache_entry_points_refuse_before_any_gpu_work():
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnCache

    def desc(**change):
        d = S(9, 16, 2, 32, sn.SN_BF16, sn.SN_CODES_INT8, 256, 256, 256, 256, 3, 6, 4, 5, 256, 256, 256, 4, 0.5, 1, 0, 256, 128, 32)
        for name, value in change.items():
            setattr(d, name, value)
        return d

    def write(d, k=256, v=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_cache_write(None if d is None else ctypes.byref(d), k, 64, 32, v, 64, 32, ws, ws_bytes, None)

    def read(d, k=256, v=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_cache_read(None if d is None else ctypes.byref(d), k, v, ws, ws_bytes, None)

    def attend(d, o=256, lse=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_cache_attend(None if d is None else ctypes.byref(d), o, lse, ws, ws_bytes, None)

    calls = (write, read, attend)
    assert all(f(None) == sn.SN_ERR_INVALID for f in calls)
    for change in ({"n_pages": 0}, {"page_size": 8}, {"page_size": 48}, {"page_size": 2048}, {"n_kv_heads": 0}, {"head_dim": 0},
                   {"head_dim": 129}, {"dtype": 2}, {"codes": 3}, {"codes": -1}, {"n_sequences": 0}, {"n_rows": -1}, {"max_rows": 7},
                   {"max_rows": 1}, {"max_pages": 0}, {"max_pages": 2 ** 27}, {"max_pages": 2 ** 26 + 1}, {"n_rows": 2 ** 30, "max_rows": 2 ** 30},
                   {"n_sequences": 65536, "n_rows": 65536}):
        d = desc(**change)
        assert lib.sn_cache_workspace_bytes(ctypes.byref(d)) == 0, change
        assert all(f(d) == sn.SN_ERR_INVALID for f in calls), change
    for change in ({"k": None}, {"v": None}, {"k": 264}, {"v": 264}, {"k_scale": None}, {"v_scale": None}, {"k_scale": 260},
                   {"row_ptr": None}, {"table": None}, {"lengths": None}):
        assert all(f(desc(**change)) == sn.SN_ERR_INVALID for f in calls), change
    for change in ({"n_heads": 0}, {"n_heads": 3}, {"n_heads": 65536}, {"causal": 2}, {"window": -1}, {"window": 3, "causal": 0},
                   {"scale": math.nan}, {"scale": math.inf}, {"q": None}, {"q": 257}):
        assert attend(desc(**change)) == sn.SN_ERR_INVALID, change
    d = desc(max_pages=2 ** 26)
    need = lib.sn_cache_workspace_bytes(ctypes.byref(d))
    assert need >= 256
    for f in calls:
        assert f(d, ws=None) == f(d, ws=128) == f(d, ws_bytes=255) == sn.SN_ERR_WORKSPACE
    assert attend(d, ws_bytes=need - 1) == sn.SN_ERR_WORKSPACE
    for f in (write, read):
        assert f(d, k=None) == f(d, v=None) == f(d, k=257) == f(d, v=257) == sn.SN_ERR_INVALID
    assert attend(d, o=None) == attend(d, o=257) == attend(d, lse=258) == sn.SN_ERR_INVALID
    empty = desc(n_rows=0, max_rows=0)
    assert write(empty, k=None) == read(empty, k=None) == attend(empty, o=None) == sn.SN_OK


# ------------------------------------------------------------------ the references themselves

@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
def test_reference_rotary_gradients_match_differences(interleaved, norm):
    """Central differences with h = 1e-6 in 64 bits: errors about h^2 and 1e-16 / h, so 1e-7 of the magnitudes."""
    gen = torch.Generator().manual_seed(3)
    x, dy = (torch.randn((5, 2, 9), generator=gen, dtype=torch.float64) for _ in range(2))
    w = torch.randn(9, generator=gen, dtype=torch.float64)
    pos = torch.tensor([[3, -4, 0, 1, 9], [1, 1, 2, 0, -5]], dtype=torch.int32)
    args = {"x": x, "w": w}

    def run(**change):
        y = {**args, **change}
        return R.rotary(y["x"], y["w"], pos, [1.0, 0.3, 0.1], [0, 1, 1], interleaved, norm, 1e-6, dy)[0]

    ref, h = run(), 1e-6
    for name in ("x", "w") if norm else ("x",):
        e = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
        ends = [(run(**{name: args[name] + s * h * e})["y"][0] * dy).sum() for s in (1, -1)]
        value, mag = ref["d" + name]
        assert abs(float(ends[0] - ends[1]) / (2 * h) - float((value * e).sum())) <= 1e-7 * float((mag * e.abs()).sum())


def test_reference_codes():
    """The smallest, the largest and ties by hand; all 127 values are their own codes; rounding is to the nearest."""
    y = R.e4m3([2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17, 19, 448, 460, -1.0625, 0.0])
    assert y.tolist() == [2.0 ** -9, 0.0, 2 * 2.0 ** -9, 16, 20, 448, 448, -1.0, 0.0]
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3(every), every)
    x = np.random.default_rng(1).uniform(-448, 448, 5000)
    near = every[np.abs(np.abs(x)[:, None] - every[None]).argmin(1)] * np.sign(x)
    assert np.array_equal(R.e4m3(x), near)
    y, scale = R.quantise(torch.tensor([[127.0, 0.5, 1.5, -2.5], [0.0, 0.0, 0.0, 0.0], [math.inf, 1, 1, 1]]), "int8")
    assert y.tolist() == [[127, 0, 2, -2], [0] * 4, [0] * 4] and scale[0] == 1 and scale[1] == 0 and math.isnan(scale[2])

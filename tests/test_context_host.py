"""CPU checks of the context operators: what the descriptors refuse, before any GPU work, the position
thresholds, and the 64-bit references against central differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import context_ref as R


def _sn():
    import os
    import schnet_cfconv_force_amd as sn
    if not os.path.exists(sn.LIB_PATH):
        from schnet_cfconv_force_amd import build
        build.build(verbose=False)
    return sn


# ------------------------------------------------------------------ thresholds

def buckets_by_distance(rel, n_buckets, far):
    """The definition, one offset at a time: halves by sign, near distances alone, then equal ratios."""
    half, near = n_buckets // 2, n_buckets // 4
    d = -rel if rel <= 0 else rel - 1
    j = d if d < near else min(half - 1, near + int(math.log(d / near) / math.log(far / near) * (half - near) + 1e-12))
    return half - 1 - j if rel <= 0 else half + j


@pytest.mark.parametrize("n_buckets,far", [(4, 2), (8, 20), (32, 128), (32, 1000), (64, 128), (16, 5)])
def test_thresholds_give_the_logarithmic_buckets(n_buckets, far):
    sn = _sn()
    thr = sn.relative_thresholds(n_buckets, far)
    assert thr.shape == (n_buckets - 1,) and thr.dtype == np.int32 and np.all(np.diff(thr) >= 0)
    rel = np.arange(-2 * far, 2 * far + 1)
    got = R.bucket(rel, thr)
    assert got.tolist() == [buckets_by_distance(int(r), n_buckets, far) for r in rel]
    assert got.min() == 0 and got.max() == n_buckets - 1


@pytest.mark.parametrize("n_buckets,far", [(5, 20), (2, 20), (66, 128), (32, 8), (32, 0), (32, 1024), (-4, 9)])
def test_thresholds_refuse(n_buckets, far):
    sn = _sn()
    with pytest.raises(sn.SnError) as e:
        sn.relative_thresholds(n_buckets, far)
    assert e.value.status == sn.SN_ERR_INVALID


# ------------------------------------------------------------------ plans and tensors

def test_plans_refuse():
    sn = _sn()
    make = lambda *a, **k: sn.CrossAttention(*a, device="cpu", **k)  # noqa: E731
    for q_ptr, k_ptr in (([0], [0]), ([1, 3], [0, 3]), ([0, 3, 2], [0, 1, 2]), ([0, 3], [0, 1, 2]), ([0, 2 ** 31], [0, 1])):
        with pytest.raises(ValueError):
            make(q_ptr, k_ptr, 4, 2, 32)
    for heads, kv, dim in ((4, 3, 32), (0, 1, 32), (4, 0, 32), (4, 2, 0), (4, 2, 129), (70000, 1, 8)):
        with pytest.raises(sn.SnError):
            make([0, 3], [0, 5], heads, kv, dim, scale=1.0)
    with pytest.raises(sn.SnError):                  # 65 buckets
        make([0, 3], [0, 5], 4, 2, 32, thresholds=np.arange(64))
    with pytest.raises(ValueError):
        make([0, 3], [0, 5], 4, 2, 32, dtype=torch.float16)
    norm = lambda *a, **k: sn.GroupNorm(*a, device="cpu", **k)  # noqa: E731
    with pytest.raises(ValueError):
        norm([0, 5, 4], 8, 2)
    with pytest.raises(ValueError):
        norm([0, 5], 8, 2, activation="gelu")
    for channels, groups in ((8, 3), (0, 1), (8, 0), (65537, 1)):
        with pytest.raises(sn.SnError):
            norm([0, 5], channels, groups)


def test_calls_refuse_tensors_that_do_not_fit():
    """The binding's checks; the tensors lie on the CPU, and none of these calls reaches the library."""
    sn = _sn()
    plan = sn.CrossAttention([0, 3], [0, 5], 4, 2, 32, thresholds=sn.relative_thresholds(), device="cpu")
    q, k = torch.zeros(3, 4, 32), torch.zeros(5, 2, 32)
    good = {"q": q, "k": k, "v": k.clone()}
    bad = [{"q": torch.zeros(3, 4, 31)}, {"q": torch.zeros(2, 4, 32)}, {"q": q.bfloat16()}, {"k": torch.zeros(5, 4, 32)},
           {"v": torch.zeros(5, 2, 64)[:, :, ::2]}, {"bias": torch.zeros(4, 31)}, {"bias": torch.zeros(4, 32).double()},
           {"q_pos": torch.zeros(3)}, {"k_pos": torch.zeros(3, dtype=torch.int32)},
           {"keep": torch.ones(5)}, {"keep": torch.ones(4, dtype=torch.bool)},
           {"keep": torch.ones(10, dtype=torch.bool)[::2]}]
    for change in bad:
        args = {"bias": None, "q_pos": None, "k_pos": None, "keep": None, **good, **change}
        with pytest.raises(ValueError):
            plan._bind(**args)
    plain = sn.CrossAttention([0, 3], [0, 5], 4, 2, 32, device="cpu")
    with pytest.raises(ValueError):                  # a bias without thresholds
        plain._bind(**good, bias=torch.zeros(4, 32), q_pos=None, k_pos=None, keep=None)
    norm = sn.GroupNorm([0, 3], 8, 2, device="cpu")
    for x, gamma in ((torch.zeros(3, 9), None), (torch.zeros(3, 16)[:, ::2], None), (torch.zeros(3, 8), torch.ones(7)),
                     (torch.zeros(3, 8), torch.ones(8).bfloat16())):
        with pytest.raises(ValueError):
            norm._bind(x, gamma, None)


# ------------------------------------------------------------------ the C entry points

def test_attention_entry_points_refuse_before_any_gpu_work():
    """Dummy addresses that a GPU call would fault on: every check runs on the host."""
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnCrossAttention
    thr = np.arange(31, dtype=np.int32)

    def desc(**change):
        d = S(2, 6, 9, 4, 5, 256, 256, 4, 2, 32, sn.SN_BF16, 0.5, 256, 256, 256, 128, 32, 64, 32, 64, 32, None, 256, 32,
              thr.ctypes.data, None, None)
        for name, value in change.items():
            setattr(d, name, value)
        return d

    def forward(d, o=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_cross_attention_forward(None if d is None else ctypes.byref(d), o, None, ws, ws_bytes, None)

    def backward(d, o=256, lse=256, d_o=256, dq=256, dk=256, dv=256, dbias=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_cross_attention_backward(ctypes.byref(d), o, lse, d_o, 128, 32, dq, dk, dv, dbias, ws, ws_bytes,
                                               None)

    assert forward(None) == sn.SN_ERR_INVALID
    down = np.array([3, 2] + [5] * 29, np.int32)
    wide = np.array([0] * 30 + [sn.SN_MAX_BUCKET_SPAN + 1], np.int32)
    for change in ({"n_segments": 0}, {"n_q": -1}, {"max_q": 7}, {"max_q": 2}, {"max_k": 4}, {"n_kv_heads": 3},
                   {"head_dim": 0}, {"head_dim": sn.SN_MAX_HEAD_DIM + 1}, {"dtype": 2}, {"n_buckets": 0},
                   {"n_buckets": sn.SN_MAX_BUCKETS + 1}, {"n_q": 2 ** 31 - 1, "max_q": 2 ** 31 - 1}):
        d = desc(**change)
        assert lib.sn_cross_attention_workspace_bytes(ctypes.byref(d)) == 0, change
        assert forward(d) == sn.SN_ERR_INVALID and backward(d) == sn.SN_ERR_INVALID, change
    for change in ({"q_ptr": None}, {"k_ptr": None}, {"q": None}, {"k": None}, {"v": None}, {"q": 257},
                   {"scale": math.nan}, {"scale": math.inf}, {"thresholds": None}, {"thresholds": down.ctypes.data},
                   {"thresholds": wide.ctypes.data}):
        assert forward(desc(**change)) == sn.SN_ERR_INVALID and backward(desc(**change)) == sn.SN_ERR_INVALID, change
    d = desc()
    need = lib.sn_cross_attention_workspace_bytes(ctypes.byref(d))
    assert need >= 256
    for ws, size in ((None, 1 << 40), (128, 1 << 40), (256, need - 1)):
        assert forward(d, ws=ws, ws_bytes=size) == sn.SN_ERR_WORKSPACE
        assert backward(d, ws=ws, ws_bytes=size) == sn.SN_ERR_WORKSPACE
    assert forward(d, o=None) == sn.SN_ERR_INVALID and forward(d, o=257) == sn.SN_ERR_INVALID
    for name in ("o", "lse", "d_o", "dq", "dk", "dv", "dbias"):
        assert backward(d, **{name: None}) == sn.SN_ERR_INVALID, name
    assert forward(desc(n_q=0, max_q=0), o=None) == sn.SN_OK          # no query rows: nothing to do


def test_norm_entry_points_refuse_before_any_gpu_work():
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnGroupNorm

    def desc(**change):
        d = S(2, 9, 5, 256, 8, 2, sn.SN_ACT_SSP, sn.SN_F32, 1e-5, 256, 8, None, None)
        for name, value in change.items():
            setattr(d, name, value)
        return d

    def forward(d, y=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_group_norm_forward(ctypes.byref(d), y, None, None, ws, ws_bytes, None)

    def backward(d, mean=256, rstd=256, dy=256, dx=256, ws=256, ws_bytes=1 << 40):
        return lib.sn_group_norm_backward(ctypes.byref(d), mean, rstd, dy, 8, dx, None, None, ws, ws_bytes, None)

    assert lib.sn_group_norm_forward(None, 256, None, None, 256, 1 << 40, None) == sn.SN_ERR_INVALID
    for change in ({"n_segments": 0}, {"n_rows": -1}, {"max_rows": 10}, {"max_rows": 4}, {"n_channels": 0},
                   {"n_groups": 3}, {"n_groups": 0}, {"dtype": 5}, {"activation": 3}, {"activation": -1}):
        d = desc(**change)
        assert lib.sn_group_norm_workspace_bytes(ctypes.byref(d)) == 0, change
        assert forward(d) == sn.SN_ERR_INVALID and backward(d) == sn.SN_ERR_INVALID, change
    for change in ({"row_ptr": None}, {"eps": 0.0}, {"eps": math.nan}, {"eps": math.inf}, {"x": None}, {"x": 258}):
        assert forward(desc(**change)) == sn.SN_ERR_INVALID and backward(desc(**change)) == sn.SN_ERR_INVALID, change
    d = desc()
    need = lib.sn_group_norm_workspace_bytes(ctypes.byref(d))
    for ws, size in ((None, 1 << 40), (16, 1 << 40), (256, need - 1)):
        assert forward(d, ws=ws, ws_bytes=size) == sn.SN_ERR_WORKSPACE
        assert backward(d, ws=ws, ws_bytes=size) == sn.SN_ERR_WORKSPACE
    assert forward(d, y=None) == sn.SN_ERR_INVALID and forward(d, y=258) == sn.SN_ERR_INVALID
    for name in ("mean", "rstd", "dy", "dx"):
        assert backward(d, **{name: None}) == sn.SN_ERR_INVALID, name


# ------------------------------------------------------------------ the references themselves

def test_reference_attention_gradients_match_differences():
    """Central differences with h = 1e-6 in 64 bits: errors about h^2 and 1e-16 / h, so 1e-7 of the magnitudes."""
    gen = torch.Generator().manual_seed(1)
    x = {n: torch.randn(s, generator=gen, dtype=torch.float64)
         for n, s in (("q", (5, 4, 3)), ("k", (9, 2, 3)), ("v", (9, 2, 3)), ("bias", (4, 6)), ("d_o", (5, 4, 3)))}
    q_ptr, k_ptr, thr = [0, 2, 2, 5], [0, 4, 6, 9], [-2, -1, 0, 1, 2]
    keep = torch.tensor([1, 1, 0, 1, 1, 1, 1, 0, 1], dtype=torch.bool)

    def run(**change):
        y = {**x, **change}
        return R.attention(y["q"], y["k"], y["v"], q_ptr, k_ptr, 0.7, y["bias"], thr, keep=keep, d_o=x["d_o"])[0]

    ref = run()
    h = 1e-6
    for name in ("q", "k", "v", "bias"):
        e = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        ends = [(run(**{name: x[name] + s * h * e})["o"][0] * x["d_o"]).sum() for s in (1, -1)]
        slope = float(ends[0] - ends[1]) / (2 * h)
        value, mag = ref["d" + name]
        assert abs(slope - float((value * e).sum())) <= 1e-7 * float((mag * e.abs()).sum())


@pytest.mark.parametrize("act", ["none", "ssp", "silu"])
def test_reference_norm_gradients_match_differences(act):
    gen = torch.Generator().manual_seed(2)
    x, dy = (torch.randn((7, 6), generator=gen, dtype=torch.float64) for _ in range(2))
    gamma, beta = (torch.randn(6, generator=gen, dtype=torch.float64) for _ in range(2))
    args = {"x": x, "gamma": gamma, "beta": beta}

    def run(**change):
        y = {**args, **change}
        return R.group_norm(y["x"], [0, 3, 3, 7], 2, 1e-5, act, y["gamma"], y["beta"], dy)[0]

    ref = run()
    h = 1e-6
    for name in args:
        e = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
        ends = [(run(**{name: args[name] + s * h * e})["y"][0] * dy).sum() for s in (1, -1)]
        value, mag = ref["d" + name]
        assert abs(float(ends[0] - ends[1]) / (2 * h) - float((value * e).sum())) <= 1e-7 * float((mag * e.abs()).sum())


def test_training_forward_needs_what_the_backward_reads():
    sn = _sn()
    lib, S = sn.lib(), sn.binding.SnCrossAttention
    for dtype, rows, lse, n_q, want in ((sn.SN_BF16, None, 256, 6, sn.SN_ERR_INVALID), (sn.SN_BF16, 256, None, 6, sn.SN_ERR_INVALID),
                                        (sn.SN_F32, None, None, 6, sn.SN_ERR_INVALID), (sn.SN_BF16, 258, 256, 6, sn.SN_ERR_INVALID),
                                        (sn.SN_BF16, None, None, 0, sn.SN_OK)):
        d = S(2, n_q, 9, min(n_q, 4), 5, 256, 256, 4, 2, 32, dtype, 0.5, 256, 256, 256, 128, 32, 64, 32, 64, 32)
        got = lib.sn_cross_attention_forward_train(ctypes.byref(d), 256, rows, lse, 256, 1 << 40, None)
        assert got == want, (dtype, rows, lse, n_q)

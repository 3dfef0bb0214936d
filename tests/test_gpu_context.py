"""GPU: cross attention with a relative position bias and group norm with an activation, against 64-bit
references (context_ref.py states how the tolerances are derived)."""
import numpy as np
import pytest

import context_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sn():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import schnet_cfconv_force_amd as sn
    sn.lib()
    return sn


def ptr(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def rows(shape, dtype, gen, layout, scale=1.0):
    """Random rows [n, h, d] in one of several memory orders, all with the same kind of values."""
    import torch
    n, h, d = shape
    x = (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)
    if layout == "plain":
        return x
    if layout == "beside":          # two tensors side by side in a row
        buf = torch.full((n, 2, h, d), float("nan"), dtype=dtype, device="cuda")
        buf[:, 1] = x
        return buf[:, 1]
    if layout == "heads_first":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    assert layout == "odd"          # odd strides and an address that only suits one element
    buf = torch.full((n * (h * (d + 1) + 3) + 1,), float("nan"), dtype=dtype, device="cuda")
    view = buf[1:].as_strided((n, h, d), (h * (d + 1) + 3, d + 1, 1), 1)
    view.copy_(x)
    return view


def attention_case(sn, lq, lk, H, Hkv, D, dtype, bias, keep, layout, seed=0, scale=None, spread=1.0, gen_pos=None):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    dt = getattr(torch, dtype)
    qp, kp = ptr(lq), ptr(lk)
    nq, nk = int(qp[-1]), int(kp[-1])
    thr = sn.relative_thresholds(32, 128) if bias is True else bias
    c = {"q": rows((nq, H, D), dt, gen, layout, spread), "k": rows((nk, Hkv, D), dt, gen, layout),
         "v": rows((nk, Hkv, D), dt, gen, layout), "d_o": rows((nq, H, D), dt, gen, layout)}
    where = {"bias": None, "q_pos": None, "k_pos": None, "keep": None}
    if bias is not False:
        where["bias"] = torch.randn((H, len(thr) + 1), generator=gen, device="cuda")
        if gen_pos == "scattered":      # any order, far beyond the thresholds, and the ends of the type
            rng = np.random.default_rng(seed)
            for n, m in (("q_pos", nq), ("k_pos", nk)):
                p = rng.integers(-300, 300, m)
                p[::7] = rng.integers(-2 ** 31, 2 ** 31, len(p[::7]))
                where[n] = torch.from_numpy(p.astype(np.int32)).cuda()
        elif gen_pos != "default":
            where["q_pos"] = torch.from_numpy(np.concatenate([np.arange(n) for n in lq] + [[]]).astype(np.int32)).cuda()
            where["k_pos"] = torch.from_numpy(np.concatenate([np.arange(n) * 2 - 1 for n in lk] + [[]]).astype(np.int32)).cuda()
    if keep:
        kept = torch.rand(nk, generator=gen, device="cuda") < (0.8 if keep != "sparse" else 0.02)
        if keep == "empty" and len(lk) > 1:
            kept[int(kp[1]):int(kp[2])] = False
        if keep == "poison":            # what lies in absent places must not be seen
            bad = [float("nan"), float("inf"), -float("inf"), float(torch.finfo(dt).min)]
            for n in ("k", "v"):
                drop = torch.nonzero(~kept).ravel()
                for i, x in enumerate(bad):
                    c[n][drop[i::4]] = x
        where["keep"] = kept
    plan = sn.CrossAttention(qp, kp, H, Hkv, D, dtype=dt, scale=scale, thresholds=None if bias is False else thr)
    clean = dict(c)
    if keep:
        for n in ("k", "v"):
            clean[n] = torch.where(where["keep"][:, None, None], c[n], torch.zeros((), dtype=dt, device="cuda"))
    ref, factor = R.attention(clean["q"], clean["k"], clean["v"], qp, kp, plan.scale, where["bias"], thr if bias is not False else None,
                              where["q_pos"], where["k_pos"], where["keep"], clean["d_o"])
    return plan, c, where, ref, factor


def attention_run(sn, plan, c, where):
    ws = sn.cross_attention_workspace(plan)
    o, saved = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, save=True, **where)
    served = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, **where)
    dq, dk, dv, dbias = sn.cross_attention_backward(plan, c["q"], c["k"], c["v"], saved, c["d_o"], ws, **where)
    assert sn.read_status(ws) == sn.SN_OK
    got = {"o": o, "served": served, "lse": saved[1], "dq": dq, "dk": dk, "dv": dv}
    return dict(got, dbias=dbias) if dbias is not None else got


def attention_check(got, ref, factor, dtype):
    import torch
    low = dtype == "bfloat16"
    for name, g in got.items():
        worst = R.check(name, g, ref["o" if name == "served" else name], factor, low and name not in ("lse", "dbias"))
        print(f"   {name}: {worst:.2g} of the tolerance", flush=True)
    # a row without keys: exact zeros
    none = torch.isinf(ref["lse"][0])
    for name in ("o", "served", "dq"):
        assert not bool(got[name].cpu()[none].any()), name


#        lq, lk, H, Hkv, D
SHAPES = [
    ([1], [1], 1, 1, 1), ([1], [269], 4, 4, 32), ([3, 1, 2], [700, 65, 5], 8, 2, 64), ([16], [1030], 4, 1, 128),
    ([33], [31], 2, 2, 16), ([32, 0, 64, 5], [64, 7, 32, 0], 2, 1, 32), ([127, 129], [65, 63], 3, 3, 40),
    ([269, 269], [271, 140], 4, 4, 32), ([256], [257], 6, 2, 80), ([70], [300], 5, 1, 20), ([300], [70], 2, 2, 128),
    ([65], [129], 2, 1, 33), ([1, 1, 1, 1], [0, 1, 2, 300], 12, 4, 64), ([40], [90], 24, 1, 8),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(v).replace(" ", "") for v in s))
def test_attention_matches_the_reference(sn, shape, dtype):
    print(f"[attention] {shape} {dtype}", flush=True)
    plan, c, where, ref, factor = attention_case(sn, *shape, dtype, True, True, "beside", seed=len(str(shape)))
    attention_check(attention_run(sn, plan, c, where), ref, factor, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("layout", ["plain", "heads_first", "odd"])
@pytest.mark.parametrize("keep", [False, "empty", "sparse", "poison"])
@pytest.mark.parametrize("few", [True, False])
def test_attention_masks_and_layouts(sn, layout, keep, few, dtype):
    print(f"[attention] {layout} keep={keep} few={few} {dtype}", flush=True)
    lq, lk = ([2, 1, 3], [150, 70, 260]) if few else ([140, 33, 75], [150, 70, 260])
    plan, c, where, ref, factor = attention_case(sn, lq, lk, 6, 2, 48, dtype, keep != "sparse", keep, layout, seed=3)
    attention_check(attention_run(sn, plan, c, where), ref, factor, dtype)


#        lq, lk, H, Hkv, D, thresholds, scale: what the shapes above do not reach
SPLIT = [
    # few key/value heads and segments: the keys of many rows are cut and joined, a segment without keys in a cut
    ([40], [1200], 2, 2, 32, True, None), ([130, 40, 33], [1800, 700, 3], 2, 1, 64, True, None), ([35], [2100], 1, 1, 128, False, None),
    # ... and the keys of few rows
    ([1], [5000], 2, 1, 64, True, None), ([9, 2], [3000, 40], 3, 3, 33, True, None),
    # many rows per key: the rows of the dk, dv pass are cut and joined
    ([700], [40], 4, 2, 32, True, None), ([700, 5], [40, 129], 4, 1, 64, True, None), ([900], [33], 3, 1, 128, False, None),
    # a table of offsets that only one or two heads of a subgroup fit
    ([20, 150], [170, 60], 6, 1, 32, "wide", None), ([3], [900], 8, 1, 64, "half", None), ([80], [90], 16, 1, 16, "half", None),
    # scales of either sign and none
    ([70, 3], [100, 40], 4, 2, 40, True, -0.3), ([70, 3], [100, 40], 2, 2, 64, True, 0.0), ([5], [700], 2, 2, 16, False, -1.0),
]
SPANS = {"wide": [-1023, -8, 1, 9, 1023], "half": [-500, -4, 0, 4, 500]}


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", SPLIT, ids=lambda s: "x".join(str(v).replace(" ", "") for v in s))
def test_attention_splits_subgroups_and_scales(sn, shape, dtype):
    print(f"[attention] {shape} {dtype}", flush=True)
    lq, lk, H, Hkv, D, thr, scale = shape
    thr = np.array(SPANS[thr], np.int32) if isinstance(thr, str) else thr
    plan, c, where, ref, factor = attention_case(sn, lq, lk, H, Hkv, D, dtype, thr, True, "plain", seed=len(str(shape)) + 50,
                                                 scale=scale)
    attention_check(attention_run(sn, plan, c, where), ref, factor, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("lq", [[3, 2, 5], [40, 33, 50], [35]], ids=str)
def test_attention_keeps_nan_where_it_belongs(sn, lq, name, dtype):
    """A NaN in a row that counts reaches exactly the outputs that depend on it, in its head and segment."""
    import torch
    print(f"[attention] NaN in {name}, rows {lq} {dtype}", flush=True)
    lk = [70, 90, 600] if len(lq) > 1 else [1100]
    plan, c, where, ref, factor = attention_case(sn, lq, lk, 4, 2, 32, dtype, False, True, "plain", seed=60)
    where["keep"][lk[0] - 1:lk[0] + 1] = True
    at = lq[0] - 1 if name == "q" else lk[0] - 1
    c[name][at, 1, 3] = float("nan")
    clean = {n: c[n] if n not in ("k", "v") else torch.where(where["keep"][:, None, None], c[n], torch.zeros_like(c[n])) for n in c}
    ref, factor = R.attention(clean["q"], clean["k"], clean["v"], plan.q_ptr.cpu().numpy(), plan.k_ptr.cpu().numpy(), plan.scale,
                              keep=where["keep"], d_o=c["d_o"])
    got = attention_run(sn, plan, c, where)
    for n, g in got.items():
        value, mag = ref["o" if n == "served" else n]
        bad = torch.isnan(value)
        assert torch.equal(torch.isnan(g.cpu()), bad), n
        fine = torch.where(bad, torch.zeros_like(value), value), torch.where(bad, torch.zeros_like(mag), mag)
        R.check(n, torch.where(bad.cuda(), torch.zeros_like(g), g), fine, factor, dtype == "bfloat16" and n != "lse")


THRESHOLDS = {"one": [], "two": [0], "equal": [-3, -3, 0, 0, 5], "wide": [-1000, -40, 0, 40, 1046],
              "many": list(range(-31, 32)), "far": [2 ** 31 - 9, 2 ** 31 - 1], "low": [-2 ** 31, -2 ** 31 + 3]}


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("where_pos", ["scattered", "default", "given"])
@pytest.mark.parametrize("thr", list(THRESHOLDS))
def test_attention_position_buckets(sn, thr, where_pos, dtype):
    print(f"[attention] thresholds {thr}, positions {where_pos} {dtype}", flush=True)
    plan, c, where, ref, factor = attention_case(sn, [130, 9], [200, 77], 4, 2, 32, dtype, np.array(THRESHOLDS[thr], np.int32),
                                                 True, "plain", seed=5, gen_pos=where_pos)
    attention_check(attention_run(sn, plan, c, where), ref, factor, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_attention_large_scores(sn, dtype):
    """Scores of both signs far beyond exp's range: the running maximum has to carry them."""
    print(f"[attention] large scores {dtype}", flush=True)
    plan, c, where, ref, factor = attention_case(sn, [70, 2], [300, 300], 2, 2, 64, dtype, False, False, "plain", seed=6,
                                                 spread=40.0)
    attention_check(attention_run(sn, plan, c, where), ref, factor, dtype)


def test_attention_offsets_beyond_32_bits(sn):
    import torch
    print("[attention] row offsets beyond 2^31 elements", flush=True)
    n, H, D, step = 6, 2, 32, 2 ** 29
    gen = torch.Generator(device="cuda").manual_seed(7)
    buf = torch.empty((n - 1) * step + H * D, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((n, H, D), (step, D, 1))
    small = torch.randn((n, H, D), generator=gen, device="cuda").to(torch.bfloat16)
    far.copy_(small)
    other = torch.randn((n, H, D), generator=gen, device="cuda").to(torch.bfloat16)
    for lengths in ([n], [2, 4]):
        plan = sn.CrossAttention(ptr(lengths), ptr(lengths), H, H, D, dtype=torch.bfloat16)
        for names in (("q", "d_o"), ("k", "v")):
            near = {m: other for m in ("q", "k", "v", "d_o")}
            near.update({m: small for m in names})
            wide = dict(near, **{m: far for m in names})
            where = {"bias": None, "q_pos": None, "k_pos": None, "keep": None}
            a, b = attention_run(sn, plan, near, where), attention_run(sn, plan, wide, where)
            for m in a:
                assert torch.equal(a[m], b[m]), (names, m)


def test_attention_repeats_bit_for_bit_on_any_stream_and_in_a_graph(sn):
    import torch
    print("[attention] streams and graphs", flush=True)
    plan, c, where, ref, factor = attention_case(sn, [200, 90], [330, 150], 4, 2, 64, "bfloat16", True, True, "plain", seed=8)
    first = attention_run(sn, plan, c, where)
    again = attention_run(sn, plan, c, where)
    ws = sn.cross_attention_workspace(plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, saved = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, save=True, stream=side, **where)
    grads = sn.cross_attention_backward(plan, c["q"], c["k"], c["v"], saved, c["d_o"], ws, stream=side, **where)
    torch.cuda.current_stream().wait_stream(side)
    for name in first:
        assert torch.equal(first[name], again[name]), name
    for name, t in zip(("o", "dq", "dk", "dv", "dbias"), (o, *grads)):
        assert torch.equal(first[name], t), name
    # recorded once, replayed on new inputs with other work in between
    live = {n: t.clone() for n, t in c.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, saved = sn.cross_attention_forward(plan, live["q"], live["k"], live["v"], ws, save=True, **where)
        grads = sn.cross_attention_backward(plan, live["q"], live["k"], live["v"], saved, live["d_o"], ws, **where)
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in live.values():
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = attention_run(sn, plan, live, where)
        for name, t in zip(("o", "dq", "dk", "dv", "dbias"), (o, *grads)):
            assert torch.equal(want[name], t), (seed, name)


@pytest.mark.parametrize("few", [True, False])
def test_attention_flags_contradicting_pointers(sn, few):
    """A device pointer array that outgrows the plan's sizes: flagged, its segment skipped, nothing out of range."""
    import torch
    print(f"[attention] contradicting pointers few={few}", flush=True)
    lq = [2, 3, 1] if few else [40, 50, 60]
    plan, c, where, ref, factor = attention_case(sn, lq, [70, 80, 90], 4, 2, 32, "float32", False, False, "plain", seed=9)
    plan.k_ptr.copy_(torch.tensor([0, 70, 300, 240], dtype=torch.int32))     # the second and third contradict
    ws = sn.cross_attention_workspace(plan)
    o, saved = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, save=True)
    assert sn.read_status(ws) == sn.SN_ERR_INVALID
    assert sn.read_status(ws) == sn.SN_OK
    R.check("o", o[:lq[0]], tuple(t[:lq[0]] for t in ref["o"]), factor, False)
    sn.cross_attention_backward(plan, c["q"], c["k"], c["v"], saved, c["d_o"], ws)
    assert sn.read_status(ws) == sn.SN_ERR_INVALID


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lq", [[3, 1], [200, 77]], ids=str)
def test_attention_of_a_single_key_has_no_score_gradient(sn, lq, dtype):
    """Whatever its score, the only key has the weight one: o is its value, dq, dk and dbias are zeros."""
    import torch
    print(f"[attention] single keys {lq} {dtype}", flush=True)
    plan, c, where, ref, factor = attention_case(sn, lq, [1, 1], 4, 2, 40, dtype, True, False, "plain", seed=61, spread=20.0)
    got = attention_run(sn, plan, c, where)
    R.check("dv", got["dv"], ref["dv"], factor, dtype == "bfloat16")
    R.check("o", got["o"], ref["o"], factor, dtype == "bfloat16")
    for name in ("dq", "dk", "dbias"):
        assert not bool(got[name].any()), name


def test_attention_gradient_matches_differences(sn):
    """Along a random direction, (L(x + h e) - L(x - h e)) / 2h of L = sum(o d_o) against <grad, e>.  With h = 2^-5
    the third-order term is below h^2 = 1e-3 of the magnitudes, the fp32 noise far below."""
    import torch
    print("[attention] differences", flush=True)
    plan, c, where, ref, factor = attention_case(sn, [90, 3], [150, 40], 4, 2, 32, "float32", True, True, "plain", seed=10)
    got = attention_run(sn, plan, c, where)
    ws = sn.cross_attention_workspace(plan)
    gen = torch.Generator(device="cuda").manual_seed(11)
    h = 2.0 ** -5
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("bias", "dbias")):
        base = where["bias"] if name == "bias" else c[name]
        e = torch.randn(base.shape, generator=gen, device="cuda")
        ends = []
        for sign in (1, -1):
            moved, at = dict(c), dict(where)
            (at if name == "bias" else moved)[name] = base + sign * h * e
            o = sn.cross_attention_forward(plan, moved["q"], moved["k"], moved["v"], ws, **at)
            ends.append(float((o.double() * c["d_o"].double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        want = float((got[grad].double() * e.double()).sum())
        mag = float((ref[grad][1].cuda() * e.double().abs()).sum())
        print(f"   {name}: {slope:.6g} against {want:.6g} (magnitudes {mag:.3g})", flush=True)
        assert abs(slope - want) <= h * h * mag


# ------------------------------------------------------------------ group norm

def norm_case(sn, lengths, C, groups, act, dtype, layout="plain", affine=True, shift=0.0, seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2000 + seed)
    dt = getattr(torch, dtype)
    p = ptr(lengths)
    n = int(p[-1])
    x = (rows((n, 1, C), torch.float32, gen, "plain")[:, 0] * 1.5 + torch.randn(C, generator=gen, device="cuda") + shift).to(dt)
    dy = rows((n, 1, C), dt, gen, layout)[:, 0]
    if layout != "plain":
        buf = rows((n, 1, C), dt, gen, layout)
        buf[:, 0] = x
        x = buf[:, 0]
    gamma = 1 + 0.3 * torch.randn(C, generator=gen, device="cuda") if affine else None
    beta = 0.3 * torch.randn(C, generator=gen, device="cuda") if affine else None
    plan = sn.GroupNorm(p, C, groups, activation=act, dtype=dt)
    ref, factor = R.group_norm(x, p, groups, 1e-5, act, gamma, beta, dy)
    return plan, x, gamma, beta, dy, ref, factor


def norm_run(sn, plan, x, gamma, beta, dy):
    ws = sn.group_norm_workspace(plan)
    y, saved = sn.group_norm_forward(plan, x, gamma, beta, ws, save=True)
    served = sn.group_norm_forward(plan, x, gamma, beta, ws)
    dx, dgamma, dbeta = sn.group_norm_backward(plan, x, gamma, beta, saved, dy, ws)
    assert sn.read_status(ws) == sn.SN_OK
    return {"y": y, "served": served, "mean": saved[0], "rstd": saved[1], "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def norm_check(got, ref, factor, dtype):
    for name, g in got.items():
        low = dtype == "bfloat16" and name in ("y", "served", "dx")
        value = ref["y" if name == "served" else name]
        worst = R.check(name, g, value, factor, low)
        print(f"   {name}: {worst:.2g} of the tolerance", flush=True)


#     lengths, channels, groups
NORMS = [
    ([1], 1, 1), ([269], 128, 8), ([269, 0, 1, 33], 128, 128), ([5, 64, 100], 96, 1), ([17, 400], 30, 10),
    ([2000], 64, 4), ([3000, 5, 1500], 24, 3), ([700, 900], 512, 32), ([0, 0], 8, 2), ([1, 2, 3], 1000, 5),
    ([50], 7, 7), ([15668], 128, 8), ([20], 2048, 2), ([9000, 40], 33, 3),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("act", ["none", "ssp", "silu"])
@pytest.mark.parametrize("shape", NORMS, ids=lambda s: "x".join(str(v).replace(" ", "") for v in s))
def test_norm_matches_the_reference(sn, shape, act, dtype):
    print(f"[norm] {shape} {act} {dtype}", flush=True)
    plan, *args, ref, factor = norm_case(sn, *shape, act, dtype, seed=len(str(shape)))
    norm_check(norm_run(sn, plan, *args), ref, factor, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("layout", ["beside", "odd"])
@pytest.mark.parametrize("shape", [([269, 40], 128, 8), ([5000], 40, 5), ([12, 7], 33, 3)], ids=str)
def test_norm_layouts_without_parameters(sn, shape, layout, dtype):
    print(f"[norm] {shape} {layout} {dtype}", flush=True)
    plan, *args, ref, factor = norm_case(sn, *shape, "silu", dtype, layout=layout, affine=False, seed=4)
    norm_check(norm_run(sn, plan, *args), ref, factor, dtype)


# groups wider than a block's vectors, whole and with short last pieces, and many short segments
WIDE = [([40, 3], 8192, 1), ([700], 4096, 1), ([30, 0, 9], 6000, 2), ([7], 65536, 1), ([300, 2], 1500, 1), ([1] * 300, 16, 4)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: f"{len(s[0])}x{max(s[0])}x{s[1]}x{s[2]}")
def test_norm_wide_groups(sn, shape, layout, dtype):
    print(f"[norm] wide {shape[1:]} {layout} {dtype}", flush=True)
    plan, *args, ref, factor = norm_case(sn, *shape, "ssp", dtype, layout=layout, seed=9)
    norm_check(norm_run(sn, plan, *args), ref, factor, dtype)


@pytest.mark.parametrize("shape", [([269, 40], 128, 8), ([6000], 64, 2)], ids=str)
def test_norm_far_from_zero(sn, shape):
    """A mean of 1000 standard deviations: the variance must not come from a difference of large sums."""
    print(f"[norm] shifted {shape}", flush=True)
    plan, *args, ref, factor = norm_case(sn, *shape, "ssp", "float32", shift=1500.0, seed=5)
    norm_check(norm_run(sn, plan, *args), ref, factor, "float32")


@pytest.mark.parametrize("rows_", [3, 5000])
def test_norm_constant_rows_give_beta(sn, rows_):
    import torch
    print(f"[norm] constant {rows_}", flush=True)
    plan = sn.GroupNorm([0, rows_], 32, 4)
    x = torch.full((rows_, 32), 0.75, device="cuda")
    beta = torch.arange(32, dtype=torch.float32, device="cuda")
    got = norm_run(sn, plan, x, None, beta, torch.ones_like(x))
    assert torch.equal(got["y"], beta.expand(rows_, 32)) and bool(torch.isfinite(got["dx"]).all())


def test_norm_of_single_elements_has_no_gradient(sn):
    """A group of one element is beta whatever x is."""
    import torch
    print("[norm] single elements", flush=True)
    plan, x, gamma, beta, dy, ref, factor = norm_case(sn, [1, 1, 1], 24, 24, "silu", "float32", seed=10)
    assert not bool(norm_run(sn, plan, x, gamma, beta, dy)["dx"].any())


def test_norm_repeats_bit_for_bit_on_any_stream_and_in_a_graph(sn):
    import torch
    print("[norm] streams and graphs", flush=True)
    for shape in (([269, 300], 128, 8), ([9000, 100], 64, 4)):
        plan, x, gamma, beta, dy, ref, factor = norm_case(sn, *shape, "ssp", "bfloat16", seed=6)
        first, again = norm_run(sn, plan, x, gamma, beta, dy), norm_run(sn, plan, x, gamma, beta, dy)
        for name in first:
            assert torch.equal(first[name], again[name]), name
        ws = sn.group_norm_workspace(plan)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y, saved = sn.group_norm_forward(plan, x, gamma, beta, ws, save=True, stream=side)
        dx, _, _ = sn.group_norm_backward(plan, x, gamma, beta, saved, dy, ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, first["y"]) and torch.equal(dx, first["dx"])
        live, grad = x.clone(), dy.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            y, saved = sn.group_norm_forward(plan, live, gamma, beta, ws, save=True)
            outs = sn.group_norm_backward(plan, live, gamma, beta, saved, grad, ws)
        for seed in range(3):
            gen = torch.Generator(device="cuda").manual_seed(seed)
            for t in (live, grad):
                t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            want = norm_run(sn, plan, live, gamma, beta, grad)
            for name, t in zip(("y", "dx", "dgamma", "dbeta"), (y, *outs)):
                assert torch.equal(want[name], t), (seed, name)


@pytest.mark.parametrize("lengths", [[40, 50, 60], [4000, 50, 3000]], ids=str)
def test_norm_flags_contradicting_pointers(sn, lengths):
    import torch
    print(f"[norm] contradicting pointers {lengths}", flush=True)
    plan, x, gamma, beta, dy, ref, factor = norm_case(sn, lengths, 32, 4, "ssp", "float32", seed=7)
    a = lengths[0]
    plan.row_ptr.copy_(torch.tensor([0, a, 10 * sum(lengths), sum(lengths)], dtype=torch.int32))
    ws = sn.group_norm_workspace(plan)
    y, saved = sn.group_norm_forward(plan, x, gamma, beta, ws, save=True)
    assert sn.read_status(ws) == sn.SN_ERR_INVALID
    R.check("y", y[:a], tuple(t[:a] for t in ref["y"]), factor, False)
    sn.group_norm_backward(plan, x, gamma, beta, saved, dy, ws)
    assert sn.read_status(ws) == sn.SN_ERR_INVALID


def test_norm_gradient_matches_differences(sn):
    """As for the attention: h = 2^-5, third-order terms below h^2 of the magnitudes."""
    import torch
    print("[norm] differences", flush=True)
    plan, x, gamma, beta, dy, ref, factor = norm_case(sn, [90, 31], 64, 4, "silu", "float32", seed=8)
    got = norm_run(sn, plan, x, gamma, beta, dy)
    ws = sn.group_norm_workspace(plan)
    gen = torch.Generator(device="cuda").manual_seed(12)
    h = 2.0 ** -5
    for k, grad in enumerate(("dx", "dgamma", "dbeta")):
        e = torch.randn((x, gamma, beta)[k].shape, generator=gen, device="cuda")
        ends = []
        for sign in (1, -1):
            args = [x, gamma, beta]
            args[k] = args[k] + sign * h * e
            y = sn.group_norm_forward(plan, *args, ws)
            ends.append(float((y.double() * dy.double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        want = float((got[grad].double() * e.double()).sum())
        mag = float((ref[grad][1].cuda() * e.double().abs()).sum())
        print(f"   {grad}: {slope:.6g} against {want:.6g} (magnitudes {mag:.3g})", flush=True)
        assert abs(slope - want) <= h * h * mag


# ------------------------------------------------------------------ the operators together

def test_context_embedding_example(sn):
    """The block begins as the identity: its rows give the plain model's energies and forces bit for bit.  Fitted, it
    explains most of its target, and the model runs on its rows."""
    import os
    import sys

    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import context_embedding as ex
    print("[example] context embedding", flush=True)
    cfg, x, states, state_ptr, target = ex.make_inputs(2)
    block = ex.ContextBlock(cfg["replica_ptr"], state_ptr, cfg["hyper"]["n_features"])
    pos = torch.from_numpy(cfg["pos"]).cuda()
    plain = ex.evaluate(sn.Model(cfg["params"], cfg["hyper"]), sn.System(cfg["replica_ptr"], cfg["types"], cfg["box"]), cfg, pos)
    with torch.no_grad():
        same = ex.evaluate(*ex.model_of_rows(cfg, block(x, states)), cfg, pos)
    assert torch.equal(plain[0], same[0]) and torch.equal(plain[1], same[1])
    losses = ex.fit(block, x, states, target, steps=100)
    print(f"   relative error {losses[-1]:.3f}", flush=True)
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]
    with torch.no_grad():
        energy, forces, ws, _ = ex.evaluate(*ex.model_of_rows(cfg, block(x, states)), cfg, pos)
    assert sn.read_status(ws) == sn.SN_OK and bool(torch.isfinite(forces).all())
    assert not torch.equal(energy, plain[0])

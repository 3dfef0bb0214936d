"""GPU: the context operators at masks, sizes and addresses where they can go wrong, against 64-bit references
(context_ref.py states how the tolerances are derived)."""
import numpy as np
import pytest

import context_ref as R
from test_gpu_context import attention_case, attention_check, attention_run, norm_case, norm_check, norm_run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sn():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import schnet_cfconv_force_amd as sn
    sn.lib()
    return sn


# ------------------------------------------------------------------ cross attention: masks in runs

MASKS = {"first32": lambda j, n: j >= 32, "first40": lambda j, n: j >= 40, "first96": lambda j, n: j >= 96,
         "alternate": lambda j, n: j // 32 % 2 == 1, "last": lambda j, n: j == n - 1}


@pytest.mark.parametrize("positions", ["default", "scattered"])
@pytest.mark.parametrize("thr", ["one", "several"])
@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("dtype,D", [("float32", 16), ("float32", 32), ("bfloat16", 40), ("bfloat16", 64), ("float32", 128)])
def test_attention_masks_in_runs_of_keys(sn, dtype, D, mask, thr, positions):
    """Absent keys in runs, with a bias: a tile whose first half has no key still takes its bias from the second."""
    import torch
    print(f"[attention] {mask} thresholds {thr} positions {positions} {dtype} {D}", flush=True)
    lk = [150, 64, 0, 129]
    bias = np.zeros(0, np.int32) if thr == "one" else True
    plan, c, where, ref, factor = attention_case(sn, [70, 3, 2, 33], lk, 4, 2, D, dtype, bias, False, "plain", seed=70,
                                                 gen_pos=positions)
    keep = np.concatenate([MASKS[mask](np.arange(n), n) for n in lk])
    where["keep"] = torch.from_numpy(keep).cuda()
    thresholds = bias if thr == "one" else sn.relative_thresholds(32, 128)
    ref, factor = R.attention(c["q"], c["k"], c["v"], plan.q_ptr.cpu().numpy(), plan.k_ptr.cpu().numpy(), plan.scale,
                              where["bias"], thresholds, where["q_pos"], where["k_pos"], where["keep"], c["d_o"])
    attention_check(attention_run(sn, plan, c, where), ref, factor, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lq", [[3, 1, 2], [200, 77, 40]], ids=str)
def test_attention_of_a_single_kept_key_has_no_score_gradient(sn, lq, dtype):
    """Of the many keys of each segment but the last the mask keeps one: its weight is one whatever its score."""
    import torch
    print(f"[attention] single kept keys {lq} {dtype}", flush=True)
    lk = [150, 90, 70]
    plan, c, where, ref, factor = attention_case(sn, lq, lk, 4, 2, 40, dtype, True, False, "plain", seed=76, spread=20.0)
    keep = torch.zeros(sum(lk), dtype=torch.bool, device="cuda")
    keep[[140, 151]] = True
    keep[240:] = True
    where["keep"] = keep
    ref, factor = R.attention(c["q"], c["k"], c["v"], plan.q_ptr.cpu().numpy(), plan.k_ptr.cpu().numpy(), plan.scale, where["bias"],
                              sn.relative_thresholds(32, 128), where["q_pos"], where["k_pos"], keep, c["d_o"])
    got = attention_run(sn, plan, c, where)
    attention_check(got, ref, factor, dtype)
    n = sum(lq[:2])
    assert not bool(got["dq"][:n].any()) and not bool(got["dk"][:240].any())
    assert bool(got["dq"][n:].any()) and bool(got["dk"][240:].any())


def attention_dense(plan, c, where, thresholds, allowed):
    """Values in 64 bits, one head of one segment at a time, over the keys that `allowed` (bias bucket [n, m], kept [m])
    leaves to each row; a row that it leaves none is zeros.  Also the root of the sum of each output's squared terms."""
    import torch
    q, k, v, g = (c[n].double().cpu() for n in ("q", "k", "v", "d_o"))
    H, G = plan.n_heads, plan.n_heads // plan.n_kv_heads
    names = {"o": q, "dq": q, "dk": k, "dv": v}
    out, rss = ({n: torch.zeros_like(t) for n, t in names.items()} for _ in range(2))
    bias = where["bias"].double().cpu()
    out["dbias"] = torch.zeros_like(bias)
    qp, kp = plan.q_ptr.tolist(), plan.k_ptr.tolist()
    for a, b, e, f in zip(qp[:-1], qp[1:], kp[:-1], kp[1:]):
        pos = [w[i:j].cpu().numpy().astype(np.int64) if w is not None else np.arange(j - i)
               for w, i, j in ((where["q_pos"], a, b), (where["k_pos"], e, f))]
        bk = torch.from_numpy(R.bucket(np.clip(pos[1][None] - pos[0][:, None], -2 ** 31, 2 ** 31 - 1), thresholds))
        keep = torch.ones(f - e, dtype=torch.bool) if where["keep"] is None else where["keep"][e:f].cpu()
        for h in range(H):
            ok = allowed(h, bk) & keep[None]
            add = torch.where(ok, bias[h][bk], torch.full((), -torch.inf, dtype=torch.float64))
            x = q[a:b, h] @ k[e:f, h // G].T * plan.scale + add
            top = x.amax(1, keepdim=True) if f > e else torch.zeros((b - a, 1), dtype=torch.float64)
            p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
            p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
            o = p @ v[e:f, h // G]
            ds = p * (g[a:b, h] @ v[e:f, h // G].T - (g[a:b, h] * o).sum(1, keepdim=True))
            for name, at, left, right, f_ in (("o", (slice(a, b), h), p, v[e:f, h // G], 1.0),
                                              ("dq", (slice(a, b), h), ds, k[e:f, h // G], plan.scale),
                                              ("dk", (slice(e, f), h // G), ds.T, q[a:b, h], plan.scale),
                                              ("dv", (slice(e, f), h // G), p.T, g[a:b, h], 1.0)):
                out[name][at] += left @ right * f_
                rss[name][at] += (left ** 2) @ (right ** 2) * f_ ** 2
            out["dbias"][h] += torch.bincount(bk.reshape(-1), ds.reshape(-1), minlength=bias.shape[1])
    return out, {n: t.sqrt() for n, t in rss.items()}


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("low", [-float("inf"), -3.4028234663852886e38, -1e9, -1e6], ids=str)
@pytest.mark.parametrize("lq,lk", [([2, 1], [300, 40]), ([150, 33], [130, 257])], ids=str)
def test_attention_biases_that_remove_keys(sn, lq, lk, low, dtype):
    """A head's buckets of a bias as low as a mask's: their keys count as absent, also where a row has no others."""
    import torch
    print(f"[attention] bias {low} {lq} {lk} {dtype}", flush=True)
    thr = np.array([-60, -20, -3, 0, 5, 40], np.int32)
    plan, c, where, _, factor = attention_case(sn, lq, lk, 4, 2, 32, dtype, thr, True, "plain", seed=77, gen_pos="default")
    removed = torch.zeros((4, 7), dtype=torch.bool)
    removed[0, [3, 4]] = True            # a band
    removed[1, 4:] = True                # later keys
    removed[2] = True                    # all: every row of the head is empty
    where["bias"] = torch.where(removed.cuda(), torch.full((), low, device="cuda"), where["bias"])
    want, rss = attention_dense(plan, c, {**where, "bias": where["bias"].masked_fill(removed.cuda(), 0.0)}, thr,
                                lambda h, bk: ~removed[h][bk])
    got = attention_run(sn, plan, c, where)
    assert torch.equal(got["o"], got["served"])
    assert bool(torch.isneginf(got["lse"][:, 2]).all()) and not bool(got["o"][:, 2].any())
    assert not bool(got["dbias"].cpu()[removed].any())
    for name, value in want.items():
        # bf16: two roundings of 2^-8 / sqrt(3) root mean square, of the output and of one operand of each term
        bound = 2.0 ** -12 if name == "dbias" or dtype == "float32" else 2.0 ** -7.5
        scale = value.norm() if name not in rss else torch.maximum(value.norm(), rss[name].norm())
        off = float((got[name].double().cpu() - value).norm() / scale)
        print(f"   {name}: {off:.2g}", flush=True)
        assert off <= bound, name


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), 3.3e38, -3.4e38], ids=str)
@pytest.mark.parametrize("lq,lk", [([2, 1], [90, 40]), ([150, 33], [130, 257]), ([40], [1200]), ([2], [2500])], ids=str)
def test_attention_of_infinite_and_huge_values(sn, lq, lk, value, dtype):
    """A kept value that is infinite, or large enough that a partial sum overflows where the result does not, reaches
    its column of its segment and head as the definition has it; nothing else changes."""
    import torch
    print(f"[attention] value {value} {lq} {lk} {dtype}", flush=True)
    thr = np.array([-60, -20, -3, 0, 5, 40], np.int32)
    plan, c, where, _, factor = attention_case(sn, lq, lk, 4, 2, 40, dtype, thr, True, "plain", seed=78, gen_pos="default")
    at = lk[0] - 7
    where["keep"][at] = True
    c["v"][at, 1, 5] = value
    want, _ = attention_dense(plan, c, where, thr, lambda h, bk: torch.ones_like(bk, dtype=torch.bool))
    got = attention_run(sn, plan, c, where)
    for name in ("o", "served"):
        x, y = got[name].double().cpu(), want["o"].to(c["q"].dtype).double()
        hit = torch.zeros_like(x, dtype=torch.bool)
        hit[:lq[0], 2:, 5] = True
        assert torch.equal(torch.isinf(x), torch.isinf(y)) and torch.equal(x[torch.isinf(x)], y[torch.isinf(y)]), name
        assert not bool(torch.isnan(x).any()), name
        fine = torch.isfinite(y)
        off = (x - want["o"]).abs()
        # beside a huge value: 2^-8 of it for a bf16 output, else the scores' errors in its weight
        bound = (2.0 ** -7 if dtype == "bfloat16" else factor) * want["o"].abs().clamp_min(1.0)
        assert bool((off <= bound)[fine].all()), (name, float((off / bound)[fine].max()))
        assert bool(hit[torch.isinf(y)].all())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lq,lk", [([2, 1], [90, 40]), ([150, 33], [130, 257]), ([40], [1200]), ([2], [2500])], ids=str)
def test_attention_of_an_infinite_key_element(sn, lq, lk, dtype):
    """A kept key with an infinite element has the score of its sign: a row it is minus infinity for passes it over, one
    it is infinity for is no number."""
    import torch
    print(f"[attention] infinite key {lq} {lk} {dtype}", flush=True)
    plan, c, where, _, factor = attention_case(sn, lq, lk, 4, 2, 40, dtype, np.array([0], np.int32), True, "plain", seed=79,
                                               gen_pos="default")
    at = lk[0] - 7
    where["keep"][at] = True
    finite = dict(c, k=c["k"].clone())
    c["k"][at, 1, 5] = -float("inf")
    got = attention_run(sn, plan, c, where)
    away = c["q"][:lq[0], 2:, 5] > 0
    assert bool(away.any()) and bool((~away).any())
    rest = dict(where, keep=where["keep"].clone())
    rest["keep"][at] = False
    want, _ = attention_dense(plan, finite, rest, [0], lambda h, bk: torch.ones_like(bk, dtype=torch.bool))
    for name in ("o", "served"):
        x = got[name].double().cpu()
        assert bool(torch.isnan(x[:lq[0], 2:][~away.cpu()]).all()), name
        assert bool(torch.isfinite(x[:lq[0], :2]).all() and torch.isfinite(x[lq[0]:]).all()), name
        fine = torch.zeros(x.shape[:2], dtype=torch.bool)
        fine[:lq[0], 2:] = away.cpu()
        off = ((x - want["o"]).abs() / want["o"].abs().clamp_min(1.0))[fine]
        assert float(off.max()) <= (2.0 ** -7 if dtype == "bfloat16" else factor), name


# ------------------------------------------------------------------ cross attention: bits of the weights

@pytest.mark.parametrize("lq,lk,D", [([70, 3], [400, 65], 64), ([150], [1300], 128), ([2, 1], [700, 300], 128), ([9], [2500], 40)],
                         ids=str)
def test_attention_weights_of_bf16_rows_keep_16_bits(sn, lq, lk, D):
    """Served or saved, o is the nearest bf16 to rows whose weights have 16 bits: each term of a row is at most 2^-17 of
    itself off, so its norm over the output is at most 2^-17 of the terms' sums of magnitudes, beside fp32 scores."""
    import torch
    print(f"[attention] 16-bit weights {lq} {lk} {D}", flush=True)
    plan, c, where, ref, factor = attention_case(sn, lq, lk, 4, 2, D, "bfloat16", True, False, "plain", seed=72)
    ws = sn.cross_attention_workspace(plan)
    o, (rows, lse) = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, save=True, **where)
    served = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, **where)
    assert torch.equal(o, rows.bfloat16()) and torch.equal(served, o)
    value, mag = ref["o"]
    off = float((rows.double().cpu() - value).norm() / mag.norm())
    print(f"   rows: {off:.2g} of the magnitudes", flush=True)
    assert off <= 2.0 ** -17 + factor


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lq,lk,H,Hkv,D", [([260, 33], [300, 129], 4, 2, 32), ([150], [400], 8, 2, 64), ([200, 90], [150, 260], 2, 2, 128),
                                           ([9, 3], [700, 500], 4, 1, 40), ([600], [70], 6, 3, 64)], ids=str)
def test_attention_distances_of_whole_tensors(sn, lq, lk, H, Hkv, D, dtype):
    """Distances by norms, which an allowance by magnitudes alone does not hold where dS cancels.  A bf16 rounding is at
    most 2^-8 / sqrt(3) of its value in the root mean square; o has its own, dq, dk and dv that and one of an operand of
    each term (dS, dS, p), independent of each other, so their squares add.  fp32: exponents below 64 are 2^-18 off."""
    import torch
    print(f"[attention] distances {lq} {lk} {H} {Hkv} {D} {dtype}", flush=True)
    thr = np.array([-60, -20, -3, 0, 5, 40], np.int32)
    plan, c, where, _, _ = attention_case(sn, lq, lk, H, Hkv, D, dtype, thr, True, "plain", seed=80, gen_pos="default")
    want, rss = attention_dense(plan, c, where, thr, lambda h, bk: torch.ones_like(bk, dtype=torch.bool))
    got = attention_run(sn, plan, c, where)
    assert torch.equal(got["o"], got["served"])
    for name in ("o", "dq", "dk", "dv"):
        value, terms = float(want[name].norm()), float(rss[name].norm())
        bound = 2.0 ** -17 * (value + terms)
        if dtype == "bfloat16":
            bound += 2.0 ** -8 * 3.0 ** -0.5 * (value if name == "o" else (value ** 2 + terms ** 2) ** 0.5)
        off = float((got[name].double().cpu() - want[name]).norm())
        print(f"   {name}: {off / bound:.2g} of the bound, {off / value:.2g} of the norm", flush=True)
        assert off <= bound, name


# ------------------------------------------------------------------ outputs at any element

@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lq,lk", [([2], [300]), ([70, 5], [130, 40]), ([40], [1200]), ([700], [40])], ids=str)
def test_attention_outputs_at_any_element(sn, lq, lk, dtype):
    """The C entry points take any element-aligned address: outputs one element beyond an aligned one hold the same bits
    (rows stored whole, key splits joined, row splits joined), and nothing beside them is written."""
    import torch
    print(f"[attention] outputs off alignment {lq} {lk} {dtype}", flush=True)
    plan, c, where, ref, factor = attention_case(sn, lq, lk, 2, 2, 32, dtype, True, True, "plain", seed=73)
    want = attention_run(sn, plan, c, where)
    ws = sn.cross_attention_workspace(plan)
    stream = torch.cuda.current_stream().cuda_stream
    op = plan._bind(c["q"], c["k"], c["v"], **where)
    got, guard = {}, 7.0

    def off(name, like, kind):
        buf = torch.full((like.numel() + 2,), guard, dtype=kind, device="cuda")
        got[name] = buf
        return buf[1:].data_ptr()

    f32 = torch.float32
    at = {"o": off("o", c["q"], plan.dtype), "lse": off("lse", want["lse"], f32), "rows": off("rows", c["q"], f32)}
    if dtype == "float32":
        at["rows"] = at["o"]
    st = sn.lib().sn_cross_attention_forward_train(op, at["o"], at["rows"], at["lse"], ws.data_ptr(), ws.numel(), stream)
    assert st == sn.SN_OK
    grads = {n: off(n, like, plan.dtype) for n, like in (("dq", c["q"]), ("dk", c["k"]), ("dv", c["v"]))}
    grads["dbias"] = off("dbias", where["bias"], f32)
    H, D = plan.n_heads, plan.head_dim
    st = sn.lib().sn_cross_attention_backward(op, at["rows"], at["lse"], c["d_o"].data_ptr(), H * D, D, grads["dq"], grads["dk"],
                                              grads["dv"], grads["dbias"], ws.data_ptr(), ws.numel(), stream)
    assert st == sn.SN_OK and sn.read_status(ws) == sn.SN_OK
    for name in ("o", "lse", "dq", "dk", "dv", "dbias"):
        assert torch.equal(got[name][1:-1].view(want[name].shape), want[name]), name
        assert float(got[name][0]) == guard and float(got[name][-1]) == guard, name


# ------------------------------------------------------------------ group norm: many long segments

@pytest.mark.parametrize("lengths,C,groups,dtype", [
    ([1500, 40] * 64, 128, 8, "float32"), ([1500, 0, 3] * 50, 128, 8, "float32"), ([5000] + [20] * 130, 512, 32, "bfloat16"),
    ([4200] + [7] * 600, 40, 5, "bfloat16"), ([1100] + [9] * 700, 33, 3, "float32")], ids=lambda v: f"{v[0]}of{len(v)}" if isinstance(v, list) else str(v))
def test_norm_backward_of_many_segments_longer_than_a_block_holds(sn, lengths, C, groups, dtype):
    """Enough segments that none of them is cut into chunks, and rows beyond what one launch holds in registers."""
    print(f"[norm] {len(lengths)} segments of up to {max(lengths)} {C} {groups} {dtype}", flush=True)
    plan, *args, ref, factor = norm_case(sn, lengths, C, groups, "ssp", dtype, seed=70)
    norm_check(norm_run(sn, plan, *args), ref, factor, dtype)


def test_norm_backward_sums_of_long_columns_keep_their_digits(sn):
    """One long segment among many, wide rows and equal addends of one sign, whose serial fp32 sum would drift by a
    multiple of its tolerance (n / 4 roundings of one direction on n rows): dbeta is n times the addend."""
    import torch
    print("[norm] long columns", flush=True)
    n, C = 12000, 2048
    plan = sn.GroupNorm(np.concatenate([[0], n + np.arange(521)]).astype(np.int32), C, 1)
    x = torch.randn((plan.n_rows, C), generator=torch.Generator(device="cuda").manual_seed(71), device="cuda")
    dy = torch.full_like(x, 0.1)
    got = norm_run(sn, plan, x, None, None, dy)
    want = plan.n_rows * float(dy[0, 0].double())
    worst = float((got["dbeta"].double() / want - 1).abs().max())
    print(f"   dbeta: {worst / (64 * R.U32):.2g} of the tolerance", flush=True)
    assert worst <= 64 * R.U32


# ------------------------------------------------------------------ streams

@pytest.mark.parametrize("what", ["attention", "norm"])
def test_a_side_stream_needs_no_wait_of_its_own(sn, what):
    """Inputs made on the current stream behind a queue of other work, whose temporaries are freed right before the
    call: the call on another stream sees the inputs, and its outputs are not written over."""
    import torch
    print(f"[streams] {what}", flush=True)
    side, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    if what == "attention":
        plan, c, where, ref, factor = attention_case(sn, [300, 90], [330, 150], 4, 2, 64, "bfloat16", True, True, "plain", seed=74)
        want = attention_run(sn, plan, c, where)
        make_ws, names = sn.cross_attention_workspace, ("q", "k", "v")
    else:
        plan, x, gamma, beta, dy, ref, factor = norm_case(sn, [900, 500], 128, 8, "ssp", "float32", seed=74)
        want = norm_run(sn, plan, x, gamma, beta, dy)
        make_ws, c, names = sn.group_norm_workspace, {"x": x}, ("x",)
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(8):
            busy = busy @ busy * 2.0 ** -12
        live = {n: c[n].clone() for n in names}
        spare = [torch.zeros_like(t) for t in live.values()]
        for t in spare:
            t.add_(busy[0, 0].to(t.dtype))
        del spare, t
        ws = make_ws(plan)
        if what == "attention":
            o, saved = sn.cross_attention_forward(plan, *(live[n] for n in names), ws, save=True, stream=side, **where)
            outs = (o, *sn.cross_attention_backward(plan, *(live[n] for n in names), saved, c["d_o"], ws, stream=side, **where))
            keys = ("o", "dq", "dk", "dv", "dbias")
        else:
            y, saved = sn.group_norm_forward(plan, live["x"], gamma, beta, ws, save=True, stream=side)
            outs = (y, *sn.group_norm_backward(plan, live["x"], gamma, beta, saved, dy, ws, stream=side))
            keys = ("y", "dx", "dgamma", "dbeta")
        del live, ws, saved
        torch.cuda.current_stream().wait_stream(side)
        for name, t in zip(keys, outs):
            assert torch.equal(want[name], t), name


# ------------------------------------------------------------------ gradients as autograd hands them

@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gradients_of_any_strides(sn, dtype):
    """The gradient of a sum is one number with strides of zero, that of a transposed use has its last index far apart."""
    import torch
    print(f"[gradients] strides {dtype}", flush=True)
    dt = getattr(torch, dtype)
    plan, c, where, _, _ = attention_case(sn, [70, 3], [65, 20], 4, 2, 32, dtype, True, False, "plain", seed=75)
    ws = sn.cross_attention_workspace(plan)
    o, saved = sn.cross_attention_forward(plan, c["q"], c["k"], c["v"], ws, save=True, **where)
    norm, x, gamma, beta, _, _, _ = norm_case(sn, [70, 3], 32, 4, "silu", dtype, seed=75)
    nws = sn.group_norm_workspace(norm)
    y, stats = sn.group_norm_forward(norm, x, gamma, beta, nws, save=True)
    for like, run in ((o, lambda g: sn.cross_attention_backward(plan, c["q"], c["k"], c["v"], saved, g, ws, **where)),
                      (y, lambda g: sn.group_norm_backward(norm, x, gamma, beta, stats, g, nws))):
        one = torch.full((), 0.5, dtype=dt, device="cuda").expand(like.shape)
        across = c["d_o"].reshape(-1)[:like.numel()].reshape(like.shape[::-1]).permute(*reversed(range(like.dim())))
        for g in (one, across):
            assert g.stride(-1) != 1
            for a, b in zip(run(g), run(g.contiguous())):
                assert torch.equal(a, b)

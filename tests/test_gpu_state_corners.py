"""GPU: the rotation of heads and the state cache at values, sizes and layouts beyond the other tests' (state_ref.py states
how the common tolerances are derived; a test with its own derives it beside it)."""
import math

import numpy as np
import pytest

import state_ref as R
from test_gpu_state import CODES, TYPES, attend_check, cache_case, kept_rows, normal, rotary_case, rotary_check, torch_type

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sn():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import schnet_cfconv_force_amd as sn
    sn.lib()
    return sn


# ------------------------------------------------------------------ bits of the weights

@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dim,heads,kv", [(32, 64, 8), (64, 64, 8), (128, 64, 8), (64, 128, 4), (128, 128, 4)])
def test_attend_weights_keep_their_bits(sn, dim, heads, kv, codes):
    """bf16 rows, three keys a sequence, scores of one product within [-1, 1]: where values cancel, the output's own rounding
    is small and an error of the weights shows.

    In u = 2^-24 of the magnitudes.  A score is exact but for log2(e) in its scale, that product and the code's scale (3 of
    the score) and the subtraction of the maximum: in powers of two at most (3 + 3) 1.45 + 2.9 = 11.6, 8.1 in p; the
    exponential 2, the code's scale in p 1, so 11.1 above and, with two additions, 12.1 below; the quotient 5, the last
    product 1, at most nine rounded additions in the matrix product: 38.2 in all.  (Weights of 16 bits are off by up to
    128.)"""
    import torch
    print(f"[attend] bits {dim} {heads}/{kv} {codes}", flush=True)
    B = 64
    c = cache_case(sn, np.ones(B, np.int64), np.full(B, 3), kv, dim, 16, "bfloat16", codes, dim + heads, heads=heads, scale=1.0)
    gen = torch.Generator(device="cuda").manual_seed(71)
    uniform = lambda *shape: (torch.rand(shape, generator=gen, device="cuda") * 2 - 1).bfloat16()     # noqa: E731
    k = torch.zeros_like(c["rows"][0])
    k[..., 0] = uniform(*k.shape[:2])
    c["rows"] = [k, c["rows"][1]]
    c["q"].zero_()
    c["q"][..., 0] = uniform(*c["q"].shape[:2])
    sn.cache_write(c["whole"], *c["rows"], c["table"], c["lengths"], c["ws"])
    o = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"])
    assert sn.read_status(c["ws"]) == sn.SN_OK
    ref, _ = R.attend(c["q"], *kept_rows(c), c["row_ptr"], c["held"], 1.0)
    print(f"worst {R.check('o', o, ref['o'], 38.2 * R.U32, True):.3f} of the tolerance", flush=True)


# ------------------------------------------------------------------ elements that do not turn

@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,pairs", [(128, 32), (128, 37), (32, 4), (32, 0), (40, 12), (40, 3), (24, 8), (20, 3), (7, 2)])
def test_rotary_elements_that_do_not_turn_keep_to_themselves(sn, dim, pairs, dtype, interleaved, norm):
    """NaN and infinities in them, in the rows and in the gradients, do not reach their neighbours."""
    import torch
    print(f"[rotary] unturned {dim} {pairs} {dtype} {interleaved} {norm}", flush=True)
    case = rotary_case(sn, 23, 3, 2, dim, [pairs] if pairs else [], interleaved, norm, dtype, 81)
    plan, q, k, positions, w, g, _, _ = case
    for i, t in enumerate((q, k, *g)):
        for r, value in ((1, math.nan), (2, math.inf), (3, -math.inf)):
            for h in range(t.shape[1]):
                t[r + 4 * i, h, 2 * pairs + (3 * r + 5 * h) % (dim - 2 * pairs)] = value
    rotary_check(sn, case, interleaved, norm, dtype)


# ------------------------------------------------------------------ scores that are not finite

@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("dim,heads,spare", [(32, 6, 2), (32, 6, 4000), (128, 36, 2)])
def test_attend_rows_of_infinite_scores(sn, dim, heads, spare, what, dtype, codes):
    """Rows all of whose scores are NaN or one infinity: the row is not a number, and its lse is what the formula gives."""
    print(f"[attend] scores {dim} {heads} {spare} {what} {dtype} {codes}", flush=True)
    c = cache_case(sn, [2, 1, 3], [40, 300, 70], 2, dim, 16, dtype, codes, 91, heads=heads, spare=spare)
    c["rows"] = [x.clone() for x in c["rows"]]
    c["rows"][0][..., 5] = c["rows"][0][..., 5].abs() + 0.5
    sn.cache_write(c["whole"], *c["rows"], c["table"], c["lengths"], c["ws"])
    for row, head in ((0, 0), (1, heads - 1), (2, 3), (5, 1)):
        c["q"][row, head, 5] = float(what)
    attend_check(sn, c)


@pytest.mark.parametrize("dtype", TYPES)
def test_attend_keys_of_minus_infinity_have_no_weight(sn, dtype):
    """Most of a long history scores -inf, whole pieces of it: the rest alone counts."""
    import torch
    c = cache_case(sn, [1, 2], [5000, 900], 1, 32, 16, dtype, None, 92, heads=3, spare=4000)
    plain = c["q"].clone()
    c["rows"] = [x.clone() for x in c["rows"]]
    low = torch.cat([torch.arange(5000) < 4100, torch.arange(900) < 300]).cuda()
    plain[..., 5], c["q"][..., 5] = 0.0, 1e30
    c["rows"][0][..., 5] = 0.0
    c["rows"][0][low, :, 5] = -1e30
    sn.cache_write(c["whole"], *c["rows"], c["table"], c["lengths"], c["ws"])
    o, lse = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"], save=True)
    assert sn.read_status(c["ws"]) == sn.SN_OK
    absent = [low[:5000].cpu().numpy(), low[5000:].cpu().numpy()]
    ref, factor = R.attend(plain, *kept_rows(c), c["row_ptr"], c["held"], c["plan"].scale, absent=absent)
    R.check("o", o, ref["o"], factor, dtype == "bfloat16")
    R.check("lse", lse, ref["lse"], 16 * R.U32)


# ------------------------------------------------------------------ many rows beside few

@pytest.mark.parametrize("codes", [None, "int8"])
@pytest.mark.parametrize("batch,longest", [(256, 65600), (65535, 20011)])
def test_rows_of_one_long_sequence_beside_many_short_ones(sn, batch, longest, codes):
    """More places of rows than a launch has blocks, of which most hold nothing."""
    import torch
    print(f"[cache] ragged {batch} {longest} {codes}", flush=True)
    counts = np.zeros(batch, np.int64)
    counts[::7] = 1
    counts[batch // 2], counts[-1] = longest, 300
    need = -(-counts // 1024)
    table = np.full((batch, int(need.max())), -1, np.int32)
    table[np.arange(table.shape[1]) < need[:, None]] = np.random.default_rng(5).permutation(int(need.sum()))
    cache = sn.StateCache(int(need.sum()), 1024, 1, 16, codes=codes)
    plan = sn.CacheRows(cache, np.concatenate([[0], np.cumsum(counts)]), table.shape[1])
    gen = torch.Generator(device="cuda").manual_seed(6)
    rows = [normal(gen, int(counts.sum()), 1, 16, to=torch.float32) for _ in range(2)]
    table, lengths, ws = torch.from_numpy(table).cuda(), torch.from_numpy(counts.astype(np.int32)).cuda(), sn.cache_workspace(plan)
    sn.cache_write(plan, *rows, table, lengths, ws)
    back = sn.cache_read(plan, table, lengths, ws)
    assert sn.read_status(ws) == sn.SN_OK
    for x, got in zip(rows, back):
        assert torch.equal(got.cpu(), R.held(x, codes).float())


# ------------------------------------------------------------------ cut histories of several row tiles

def poisoned(sn, c, b, at):
    """Values and keys of sequence b near its end that are no numbers: v NaN, k NaN and v infinite (codes hold rows of
    those as NaN)."""
    c["rows"] = [x.clone() for x in c["rows"]]
    first = int(c["ptr"][b])
    c["rows"][1][first + at[0], 0, 3] = math.nan
    c["rows"][0][first + at[1], -1, 7] = math.nan
    c["rows"][1][first + at[2], -1, 5] = math.inf
    sn.cache_write(c["whole"], *c["rows"], c["table"], c["lengths"], c["ws"])


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("causal,odd", [(True, False), (True, True), (False, False)])
def test_attend_ragged_prompts_over_shared_blocks(sn, causal, odd, dim, dtype, codes):
    """A prompt of many row tiles (two a block, or one) beside single rows and none, in a table with room: sequences that
    have fewer row tiles than the longest, on one line of tiles; also with values that some rows of a tile do not see."""
    print(f"[attend] prompts {causal} {odd} {dim} {dtype} {codes}", flush=True)
    new, held = [64, 1, 0, 5], [700, 300, 33, 70] if causal else [700, 0, 33, 3]
    c = cache_case(sn, new, held, 2, dim, 16, dtype, codes, 101, heads=32, spare=4000, causal=causal)
    if odd:
        poisoned(sn, c, 0, (690, 696, 680))
    attend_check(sn, c)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("window,odd", [(0, False), (8000, False), (8000, True)])
def test_attend_ragged_rows_over_long_histories(sn, window, odd, dim, dtype, codes):
    """A few rows of shared heads, three row tiles of the longest: units cut anywhere, with a window and without."""
    print(f"[attend] ragged {window} {odd} {dim} {dtype} {codes}", flush=True)
    c = cache_case(sn, [5, 1, 0, 3], [9000, 100, 50, 8500], 2, dim, 16, dtype, codes, 102, heads=16, spare=40, window=window)
    if odd:
        poisoned(sn, c, 0, (8997, 8998, 8996))
    attend_check(sn, c)


@pytest.mark.parametrize("batch,longest,heads,dim,dtype,codes", [(1, 150000, 3, 32, "float32", None), (1, 150000, 2, 32, "float32", "int8"),
                                                                 (1, 290000, 1, 32, "bfloat16", None), (256, 120000, 32, 64, "bfloat16", None),
                                                                 (256, 120000, 32, 64, "bfloat16", "e4m3")])
def test_attend_one_history_over_all_blocks(sn, batch, longest, heads, dim, dtype, codes):
    """More pieces of a unit than the join takes at a time."""
    print(f"[attend] pieces {batch} {longest} {heads} {dim} {dtype} {codes}", flush=True)
    held = np.random.default_rng(103).integers(1, 40, batch)
    held[batch // 3] = longest
    c = cache_case(sn, np.ones(batch, np.int64), held, 1, dim, 16, dtype, codes, 103, heads=heads)
    attend_check(sn, c)


# ------------------------------------------------------------------ angles

def test_rotary_sines_near_half_turns(sn):
    """Rows (1, 0) turn to (cos t, sin t), t = -3000 .. 3000 radians: 355 and its multiples lie close to half turns, where a
    sine is small and the angle's rounding to fp32 would show.

    In u = 2^-24: sine and cosine 8 of their own value, the second turn's addition 1, and its part of the other one at most
    2 of 2^-26 turns, 1e-14; the angle itself, in fp64, 2 roundings of 478 turns, 7e-13 radians."""
    import torch
    n = 6001
    q = torch.zeros(n, 1, 2, device="cuda")
    q[..., 0] = 1.0
    at = torch.arange(-3000, 3001, dtype=torch.int32, device="cuda")
    plan = sn.HeadRotary(n, 1, 2, freqs=[1.0], norm=False)
    y, _ = sn.head_rotary_forward(plan, q, None, at[None], sn.head_rotary_workspace(plan))
    t = at.cpu().double()
    want = torch.stack([torch.cos(t), torch.sin(t)], -1)[:, None]
    bound = 9 * R.U32 * want.abs() + 1e-12
    worst = float(((y.cpu().double() - want).abs() / bound).max())
    print(f"worst {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1


# ------------------------------------------------------------------ layouts and sizes

@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["joined", "odd"])
@pytest.mark.parametrize("dim,spare", [(16, 2), (32, 4000), (40, 2), (128, 2)])
def test_attend_strided_queries(sn, dim, spare, layout, dtype, codes):
    """Queries that are a part of wider rows, or begin at odd elements; one row of NaN among them, which is formed apart."""
    import torch
    print(f"[attend] strides {dim} {spare} {layout} {dtype} {codes}", flush=True)
    c = cache_case(sn, [3, 1, 0, 2], [150, 40, 9, 700], 2, dim, 16, dtype, codes, 111, heads=6, spare=spare)
    n, to = c["q"].shape[0], c["q"].dtype
    if layout == "joined":
        wide = torch.zeros(n, 6 + 4, dim, dtype=to, device="cuda")[:, :6]
    else:
        wide = torch.zeros(n * 6 * (dim + 1) + 1, dtype=to, device="cuda")[1:].view(n, 6, dim + 1)[..., :dim]
    wide.copy_(c["q"])
    wide[3, 2, dim - 1] = math.nan
    c["q"] = wide
    attend_check(sn, c)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kv,dim", [(300, 16), (70, 128), (33, 40)])
def test_many_heads(sn, kv, dim, dtype, codes):
    """More heads than a block has groups of lanes: written, read back and attended to."""
    import torch
    print(f"[cache] heads {kv} {dim} {dtype} {codes}", flush=True)
    c = cache_case(sn, [2, 1], [20, 37], kv, dim, 16, dtype, codes, 112)
    k, v = sn.cache_read(c["whole"], c["table"], c["lengths"], c["ws"])
    for x, got in zip(c["rows"], (k, v)):
        assert torch.equal(got.cpu(), R.held(x, codes).to(torch.float32).to(x.dtype))
    attend_check(sn, c)


@pytest.mark.parametrize("heads,kv", [(2, 300), (300, 2), (1, 65)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rotary_many_heads(sn, heads, kv, dtype):
    print(f"[rotary] heads {heads} {kv} {dtype}", flush=True)
    rotary_check(sn, rotary_case(sn, 600, heads, kv, 32, [8, 4], False, True, dtype, 113), False, True, dtype)


def test_rows_beyond_31_bits(sn):
    """Row tensors of more than 2^31 elements: turned, with their weights' gradients, written and read back."""
    import torch
    rows, heads, dim = 2 ** 21 + 5, 8, 128
    gen = torch.Generator(device="cuda").manual_seed(114)
    x = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    freqs, axes = sn.rotary_frequencies([32])
    plan = sn.HeadRotary(rows, heads, dim, freqs=freqs, axes=axes, dtype=torch.bfloat16)
    at = torch.arange(rows, dtype=torch.int32, device="cuda")[None]
    ws = sn.head_rotary_workspace(plan)
    y, _ = sn.head_rotary_forward(plan, x, None, at, ws)
    dx, _, dw, _ = sn.head_rotary_backward(plan, x, None, at, y, None, ws)
    for part in (slice(0, 40), slice(rows - 40, rows)):
        ref, factor = R.rotary(x[part], None, at[:, part], freqs, axes, False, True, 1e-6, y[part])
        R.check("y", y[part], ref["y"], factor, True)
        R.check("dx", dx[part], ref["dx"], factor, True)
    # turned back, y is its own rows but for its rounding: dw is close to sum xh^2, all positive
    want = torch.zeros(dim, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 1 << 16):
        p = slice(i, min(i + (1 << 16), rows))
        xd, g = x[p].double(), y[p].double()
        t = at[0, p, None].double() * torch.from_numpy(freqs).cuda()
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        a, b = g[..., :32].clone(), g[..., 32:64].clone()
        g[..., :32], g[..., 32:64] = a * c + b * s, b * c - a * s
        want += (g * xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-6)).sum((0, 1))
    R.check("dw", dw, (want.cpu(), 2 * want.abs().cpu()), 64 * R.U32)
    del dx, y
    page = 1024
    cache = sn.StateCache(-(-rows // page), page, heads, dim, dtype=torch.bfloat16)
    keep = sn.CacheRows(cache, [0, rows], cache.n_pages)
    table = torch.randperm(cache.n_pages, generator=gen, device="cuda").to(torch.int32)[None]
    lengths, ws = torch.tensor([rows], dtype=torch.int32, device="cuda"), sn.cache_workspace(keep)
    sn.cache_write(keep, x, x, table, lengths, ws)
    k, v = sn.cache_read(keep, table, lengths, ws)
    assert sn.read_status(ws) == sn.SN_OK and torch.equal(k, x) and torch.equal(v, x)
    q = normal(gen, 1, heads, dim, to=torch.bfloat16)
    one = sn.CacheRows(cache, [0, 1], cache.n_pages, window=100)
    o = sn.cache_attend(one, q, table, lengths, sn.cache_workspace(one))
    last = x[-100:].double().cpu()
    ref, factor = R.attend(q, [last], [last], [0, 1], [100], one.scale)
    R.check("o", o, ref["o"], factor, True)


# ------------------------------------------------------------------ long sums

@pytest.mark.parametrize("rows", [64, 5000])
def test_rotary_weight_sums_keep_their_digits(sn, rows):
    """Heads of +-1 have a norm of 1, so that a weight's gradient is the sum of exact numbers: each a little above 1, by half
    of what one step of an fp32 sum near 200 is.  A few terms of a thread, a block's sum rounded once, the sum of all: at most
    4 u of the whole."""
    import torch
    plan = sn.HeadRotary(rows, 4, 8, n_kv_heads=4, eps=1e-30)
    x = torch.ones(rows, 4, 8, device="cuda")
    x[..., ::2] = -1.0
    dy = x * (1 + 0.49 * 2.0 ** -16)
    ws = sn.head_rotary_workspace(plan)
    _, _, dqw, dkw = sn.head_rotary_backward(plan, x, x, None, dy, dy, ws)
    want = (dy.double() * x.double()).sum((0, 1)).cpu()
    for got in (dqw, dkw):
        worst = float(((got.cpu().double() - want).abs() / want).max()) / R.U32
        print(f"off by {worst:.2f} u", flush=True)
        assert worst <= 4

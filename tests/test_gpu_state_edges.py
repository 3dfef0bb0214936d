"""GPU: the rotation of heads and the state cache at masks, values, sizes and addresses where they can go wrong, and run
together as a step of new rows runs them (state_ref.py states how the tolerances are derived)."""
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


def slots(c, b, positions):
    """Page and place of positions of sequence b."""
    table, page = c["table"].cpu().numpy(), c["cache"].page_size
    p = np.asarray(positions)
    return table[b, p // page].astype(np.int64), p % page


# ------------------------------------------------------------------ values in places that no row sees

@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [16, 32, 64, 128])
@pytest.mark.parametrize("spare", [1, 4000])
def test_attend_places_that_no_row_sees(sn, dim, dtype, codes, spare):
    """NaN behind the sequences' ends, in front of the window and in pages that are nobody's: they reach nothing."""
    import torch
    print(f"[attend] unseen {dim} {dtype} {codes} {spare}", flush=True)
    c = cache_case(sn, [1, 2, 1], [5, 300, 47], 2, dim, 32, dtype, codes, 21, heads=4, window=30, spare=spare)
    want = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"]).clone()
    cache = c["cache"]
    seen = torch.zeros((cache.n_pages, cache.page_size), dtype=torch.bool)
    for b, n in enumerate(c["held"]):
        pages, at = slots(c, b, np.arange(max(0, n - int(np.diff(c["row_ptr"])[b]) + 1 - 30), n))
        seen[pages, at] = True
    unseen = ~seen[:, None].expand(-1, 2, -1).cuda()
    for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if codes is None:
            pool[unseen] = math.nan
        else:
            pool.view(torch.int8)[unseen] = 0x7f     # of e4m3 NaN
            scale[unseen] = math.nan
    got = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"])
    assert sn.read_status(c["ws"]) == sn.SN_OK
    assert torch.equal(got, want)
    attend_check(sn, c)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("spare", [1, 4000])
def test_attend_values_that_some_rows_do_not_see(sn, what, dtype, spare):
    """Rows ahead hold NaN or infinities in keys and values: rows in front of them do not see them, the others give what
    the formulas give."""
    import torch
    print(f"[attend] seen by some {what} {dtype} {spare}", flush=True)
    c = cache_case(sn, [4, 3], [70, 300], 2, 32, 16, dtype, None, 22, heads=6, spare=spare)
    for b, at, which in ((0, 68, "v"), (1, 299, "v"), (1, 298, "k")):
        page, place = slots(c, b, [at])
        pool = c["cache"].v if which == "v" else c["cache"].k
        pool[int(page[0]), 0, int(place[0]), 3] = float(what)
        c["rows"][which == "v"][int(c["ptr"][b]) + at, 0, 3] = float(what)
    attend_check(sn, c)


@pytest.mark.parametrize("dtype", TYPES)
def test_attend_infinite_and_huge_values(sn, dtype):
    """Values near the type's end whose weighted sum passes it before the division, and infinities that every row sees."""
    import torch
    c = cache_case(sn, [1, 1, 1], [200, 300, 40], 1, 32, 16, dtype, None, 23, heads=3)
    big = torch.finfo(torch_type(dtype)).max * 0.75
    for b, value in ((0, big), (1, math.inf), (2, -big)):
        p, at = slots(c, b, np.arange(0, c["held"][b], 1 if b != 1 else 7))
        c["cache"].v[torch.from_numpy(p).cuda(), 0, torch.from_numpy(at).cuda(), 5] = value
        rows = np.arange(int(c["ptr"][b]), int(c["ptr"][b + 1]), 1 if b != 1 else 7)
        c["rows"][1][torch.from_numpy(rows).cuda(), 0, 5] = value
    attend_check(sn, c)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_rows_of_nan_stay_by_themselves(sn, dtype, codes):
    import torch
    c = cache_case(sn, [3, 2], [90, 40], 2, 64, 16, dtype, codes, 24, heads=8)
    want = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"]).clone()
    c["q"][1, 5, 7] = math.nan
    got = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"])
    assert bool(torch.isnan(got[1, 5]).all())
    got[1, 5] = want[1, 5]
    assert torch.equal(got, want)


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_a_row_of_nan_written_reaches_the_rows_that_see_it(sn, codes):
    import torch
    c = cache_case(sn, [2], [50], 1, 32, 16, "float32", codes, 25, heads=2)
    one = sn.CacheRows(c["cache"], [0, 1], c["plan"].max_pages)
    row = torch.zeros((1, 1, 32), device="cuda")
    row[0, 0, 9] = math.nan
    sn.cache_write(one, torch.zeros_like(row), row, c["table"], c["lengths"], sn.cache_workspace(one))      # position 49
    got = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"])
    assert bool(torch.isfinite(got[0]).all()) and bool(torch.isnan(got[1]).all())


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_a_value_counts_whatever_its_weight(sn, what, dtype, codes):
    """A seen key whose weight is below fp32 (its score is 200 under the others): its NaN or infinity reaches the row."""
    import torch
    if codes is not None and what == "inf":
        what = "nan"        # such a row is kept as NaN
    to = torch_type(dtype)
    c = cache_case(sn, [1], [70], 1, 32, 16, dtype, codes, 38, heads=1)
    rows = [x.clone() for x in c["rows"]]
    q = c["q"]
    q[0, 0] = 1.0
    rows[0].zero_()
    rows[0][40, 0] = -200 * 32 ** 0.5 / 32
    rows[1][40, 0, 3] = float(what)
    sn.cache_write(c["whole"], rows[0], rows[1], c["table"], c["lengths"], c["ws"])
    got = sn.cache_attend(c["plan"], q, c["table"], c["lengths"], c["ws"])[0, 0]
    assert sn.read_status(c["ws"]) == sn.SN_OK and got.dtype == to
    hit = torch.isnan(got) if what == "nan" else torch.isinf(got)
    assert bool(hit.all() if codes is not None else hit[3]) and bool(codes is not None or torch.isfinite(torch.cat([got[:3], got[4:]])).all())


def test_rotary_nan_stays_in_its_head(sn):
    import torch
    plan, q, k, positions, w, g, freqs, axes = rotary_case(sn, 20, 4, 2, 32, [8, 8], False, True, "bfloat16", 26)
    ws = sn.head_rotary_workspace(plan)
    want = [t.clone() for t in sn.head_rotary_forward(plan, q, k, positions, ws, *w)]
    q[3, 2, 1], k[7, 1, 30] = math.nan, math.inf
    got = sn.head_rotary_forward(plan, q, k, positions, ws, *w)
    assert bool(torch.isnan(got[0][3, 2]).all()) and bool(torch.isnan(got[1][7, 1]).any())
    got[0][3, 2], got[1][7, 1] = want[0][3, 2], want[1][7, 1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,heads,kv,dim", [(1, 4, 4, 32), (64, 4, 4, 32), (65, 4, 4, 32), (64, 2, 4, 32), (9, 6, 1, 40), (4, 32, 8, 128),
                                               (17, 8, 8, 128), (300, 1, 1, 7), (1, 300, 1, 16), (2000, 1, 1, 2), (3, 4, 0, 32)])
def test_rotary_weight_sums_of_few_and_more_rows(sn, rows, heads, kv, dim, dtype):
    """The weights' gradients on both sides of what one block sums alone, the same with either left out, in a workspace that
    holds what was there before."""
    import torch
    case = rotary_case(sn, rows, heads, kv, dim, [dim // 2], False, True, dtype, 61)
    rotary_check(sn, case, False, True, dtype)
    plan, q, k, positions, w, g, _, _ = case
    k, g[1] = (k, g[1]) if kv else (None, None)
    ws = sn.head_rotary_workspace(plan)
    want = sn.head_rotary_backward(plan, q, k, positions, *g, ws, *w)
    ws[256:] = 255              # behind the status words
    op = plan._bind(q, k, positions, *w)
    gs, gh, ks, kh = plan._rows(*g, ("d_q", "d_k"))
    pointer = lambda t: None if t is None else t.data_ptr()
    for with_q, with_k in ((True, True), (True, False), (False, True), (False, False)):
        dq, dk = torch.empty_like(want[0]), (torch.empty_like(want[1]) if kv else None)
        sums = torch.full((2, 3 * dim), math.nan, device="cuda")
        places = [sums[i, dim:2 * dim] if on else None for i, on in enumerate((with_q, with_k))]
        st = sn.lib().sn_head_rotary_backward(op, g[0].data_ptr(), gs, gh, pointer(g[1]), ks, kh, dq.data_ptr(), pointer(dk),
                                              pointer(places[0]), pointer(places[1]), ws.data_ptr(), ws.numel(),
                                              torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == sn.SN_OK and torch.equal(dq, want[0]) and (not kv or torch.equal(dk, want[1]))
        for i, place in enumerate(places):
            if place is not None:
                assert torch.equal(place, want[2 + i] if want[2 + i] is not None else torch.zeros_like(place))
                place.fill_(math.nan)
        assert bool(torch.isnan(sums).all())


# ------------------------------------------------------------------ arrays that contradict the sizes

@pytest.mark.parametrize("codes", [None, "int8"])
@pytest.mark.parametrize("spare", [2, 4000])
@pytest.mark.parametrize("what", ["negative", "beyond", "short", "pointer"])
def test_contradicting_sequences_are_skipped_and_flagged(sn, what, codes, spare):
    import torch
    print(f"[cache] contradiction {what} {codes} {spare}", flush=True)
    c = cache_case(sn, [1, 3, 2], [20, 70, 33], 2, 32, 16, "float32", codes, 27, heads=4, spare=spare)
    plan, ws = c["plan"], c["ws"]
    want = sn.cache_attend(plan, c["q"], c["table"], c["lengths"], ws).clone()
    back = [t.clone() for t in sn.cache_read(plan, c["table"], c["lengths"], ws)]
    lengths = c["lengths"].clone()
    if what == "pointer":
        plan.row_ptr[1:3] = torch.tensor([5, 4], dtype=torch.int32)      # rows 0..4, then a negative count, then 4, 5
    else:
        lengths[1] = {"negative": -5, "beyond": plan.max_pages * 16 + 1, "short": 2}[what]
    pool = [t.clone() for t in (c["cache"].k, c["cache"].v)]
    for call, mark in ((lambda: sn.cache_attend(plan, c["q"], c["table"], lengths, ws), want),
                       (lambda: sn.cache_read(plan, c["table"], lengths, ws)[0], back[0])):
        got = call()
        assert sn.read_status(ws) == sn.SN_ERR_INVALID
        if what != "pointer":
            assert torch.equal(got[:1], mark[:1]) and torch.equal(got[4:], mark[4:])
        else:
            assert torch.equal(got[4:], mark[4:])
    rows = [torch.ones(6, 2, 32, device="cuda") for _ in range(2)]
    sn.cache_write(plan, rows[0], rows[1], c["table"], lengths, ws)
    assert sn.read_status(ws) == sn.SN_ERR_INVALID
    p, at = slots(c, 1, np.arange(70))
    for before, now in zip(pool, (c["cache"].k, c["cache"].v)):
        assert torch.equal(before[p, :, at], now[p, :, at])             # the skipped sequence's rows are as they were
    assert sn.read_status(ws) == sn.SN_OK


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("spare", [2, 4000])
def test_bad_pages_are_absent(sn, bad, codes, spare):
    """Their keys are absent, their rows read back as zeros and are not written; the workspace's status tells."""
    import torch
    print(f"[cache] bad page {bad} {codes} {spare}", flush=True)
    c = cache_case(sn, [1, 2], [100, 70], 2, 32, 16, "float32", codes, 28, heads=4, spare=spare)
    c["table"][0, 2] = bad          # positions 32 .. 47
    absent = [np.zeros(100, bool), np.zeros(70, bool)]
    absent[0][32:48] = True
    attend_check(sn, c, absent=absent, status=sn.SN_ERR_INVALID)
    pool = [t.clone() for t in c["cache"].tensors]
    k, v = sn.cache_read(c["whole"], c["table"], c["lengths"], c["ws"])
    assert sn.read_status(c["ws"]) == sn.SN_ERR_INVALID
    for got, kept in zip((k, v), kept_rows(c)):
        want = torch.cat(kept).float()
        want[32:48] = 0
        assert torch.equal(got.cpu(), want)
    sn.cache_write(c["whole"], c["rows"][0], c["rows"][1], c["table"], c["lengths"], c["ws"])
    assert sn.read_status(c["ws"]) == sn.SN_ERR_INVALID
    assert all(torch.equal(a, b) for a, b in zip(pool, c["cache"].tensors))


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("codes", [None, "e4m3"])
def test_offsets_beyond_31_bits(sn, codes):
    """Pages whose rows lie more than 2^31 elements from the first."""
    import torch
    kv, dim, page = 8, 128, 256
    per = kv * dim * page
    n_pages = 2 ** 31 // per + 40
    cache = sn.StateCache(n_pages, page, kv, dim, dtype=torch.bfloat16, codes=codes)
    gen = torch.Generator(device="cuda").manual_seed(29)
    n = 3 * page - 20
    table = torch.tensor([[n_pages - 1, 0, n_pages - 30]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    rows = [normal(gen, n, kv, dim, to=torch.bfloat16) for _ in range(2)]
    whole = sn.CacheRows(cache, [0, n], 3)
    ws = sn.cache_workspace(whole)
    sn.cache_write(whole, rows[0], rows[1], table, lengths, ws)
    k, v = sn.cache_read(whole, table, lengths, ws)
    for x, got in zip(rows, (k, v)):
        assert torch.equal(got.cpu(), R.held(x, codes).float().bfloat16())
    plan = sn.CacheRows(cache, [0, 1], 3, n_heads=16)
    c = {"plan": plan, "q": normal(gen, 1, 16, dim, to=torch.bfloat16), "table": table, "lengths": lengths, "codes": codes,
         "ws": sn.cache_workspace(plan), "rows": rows, "ptr": np.array([0, n]), "row_ptr": np.array([0, 1]), "held": [n],
         "dtype": "bfloat16"}
    attend_check(sn, c)


def test_many_sequences(sn):
    """More sequences than a wavefront has lanes and a launch has blocks on the card, most of them short."""
    rng = np.random.default_rng(30)
    held = rng.integers(1, 40, 2000)
    attend_check(sn, cache_case(sn, np.ones(2000, np.int64), held, 2, 16, 16, "float32", None, 30, heads=2))


def test_sequences_may_share_pages_and_calls_repeat_their_bits(sn):
    import torch
    for spare in (2, 4000):
        c = cache_case(sn, [1, 1, 1], [200, 160, 640], 2, 64, 32, "bfloat16", "e4m3", 31, heads=16, spare=spare)
        c["table"][1, :5] = c["table"][0, :5]       # the first 160 positions of both
        k, v = kept_rows(c)
        first = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"])
        for _ in range(5):
            assert torch.equal(sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"]), first)
        ref, factor = R.attend(c["q"], [k[0], k[0][:160], k[2]], [v[0], v[0][:160], v[2]], c["row_ptr"], c["held"], c["plan"].scale)
        R.check("o", first, ref["o"], factor, True, 2.0 ** -16)


def test_parts_over_different_keys_join_by_their_sums(sn):
    """Two halves of a history in two caches, joined by lse, are the whole."""
    import torch
    c = cache_case(sn, [1, 1], [500, 320], 2, 32, 16, "float32", None, 32, heads=4, causal=False)
    o, lse = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"], save=True)
    half = c["lengths"] // 32 * 16
    parts = [sn.cache_attend(c["plan"], c["q"], c["table"], half, c["ws"], save=True)]
    moved = torch.zeros_like(c["table"])
    for b in range(2):
        n = int(half[b]) // 16
        moved[b, :c["table"].shape[1] - n] = c["table"][b, n:]
    parts.append(sn.cache_attend(c["plan"], c["q"], moved, c["lengths"] - half, c["ws"], save=True))
    w = torch.softmax(torch.stack([p[1] for p in parts]).double(), 0)
    joined = sum(p[0].double() * a[..., None] for p, a in zip(parts, w))
    # each side is within its own tolerance of the same sums: 128 u (1 + smax / 8) of magnitudes below 8
    assert float((joined - o.double()).abs().max()) <= 2 * 128 * R.U32 * 4 * 8
    assert float((torch.logsumexp(torch.stack([p[1] for p in parts]).double(), 0) - lse.double()).abs().max()) <= 64 * R.U32 * 40


# ------------------------------------------------------------------ streams, graphs, devices

def test_calls_on_another_stream(sn):
    import torch
    c = cache_case(sn, [2, 1], [300, 80], 2, 32, 16, "float32", "int8", 33, heads=4, spare=4000)
    want = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"]).clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        q = torch.zeros_like(c["q"])
        q.copy_(c["q"], non_blocking=True)      # on its way on the current stream
        got = sn.cache_attend(c["plan"], q, c["table"], c["lengths"], c["ws"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
    plan, q, k, positions, w, g, _, _ = rotary_case(sn, 500, 4, 2, 32, [8, 8], False, True, "float32", 34)
    ws = sn.head_rotary_workspace(plan)
    want = sn.head_rotary_backward(plan, q, k, positions, *g, ws, *w)
    got = sn.head_rotary_backward(plan, q, k, positions, *g, ws, *w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("spare", [2, 4000])
def test_a_step_captured_and_replayed(sn, spare):
    """Rotation, write, read and attention of new rows in two graphs that share workspaces, replayed in turn with eager
    work between; lengths and rows change between the replays."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(35)
    B, H, kv, dim, page, max_pages = 3, 4, 2, 32, 16, 8 + spare
    cache = sn.StateCache(B * 8, page, kv, dim, codes="e4m3")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, :8] = torch.randperm(B * 8, generator=gen, device="cuda").view(B, 8).to(torch.int32)
    plan = sn.CacheRows(cache, np.arange(B + 1), max_pages, n_heads=H)
    freqs, axes = sn.rotary_frequencies([8, 8])
    turn = sn.HeadRotary(B, H, dim, n_kv_heads=kv, freqs=freqs, axes=axes)
    ws, turn_ws = sn.cache_workspace(plan), sn.head_rotary_workspace(turn)
    lengths = torch.tensor([1, 40, 100], dtype=torch.int32, device="cuda")
    qkv = torch.zeros(B, H + 2 * kv, dim, device="cuda")
    positions = torch.zeros(2, B, dtype=torch.int32, device="cuda")
    dy = normal(gen, B, H, dim, to=torch.float32), normal(gen, B, kv, dim, to=torch.float32)

    def step():
        q, k = sn.head_rotary_forward(turn, qkv[:, :H], qkv[:, H:H + kv], positions, turn_ws)
        grads = sn.head_rotary_backward(turn, qkv[:, :H], qkv[:, H:H + kv], positions, *dy, turn_ws)
        sn.cache_write(plan, k, qkv[:, H + kv:], table, lengths, ws)
        return (*sn.cache_read(plan, table, lengths, ws), sn.cache_attend(plan, q, table, lengths, ws), *grads)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for i in range(6):
        qkv.copy_(normal(gen, *qkv.shape, to=torch.float32))
        positions.fill_(i * 1000)
        graph, out = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(step(), got):
            assert torch.equal(a, b)
        lengths += 1
    assert sn.read_status(ws) == sn.SN_OK


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
def test_a_history_that_grows_row_by_row(sn, dtype, codes):
    """Rows come one (then a few) at a time, are normed and turned by (frame, residue), kept and attended to: every step
    equals attention over all rows so far, each turned by its own position."""
    import torch
    print(f"[step] {dtype} {codes}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(36)
    to = torch_type(dtype)
    B, H, kv, dim, page = 3, 6, 2, 32, 16
    cache = sn.StateCache(24, page, kv, dim, dtype=to, codes=codes)
    table = torch.randperm(24, generator=gen, device="cuda").view(B, 8).to(torch.int32)
    freqs, axes = sn.rotary_frequencies([8, 8])
    w = [normal(gen, dim, to=torch.float32) for _ in range(2)]
    kept = [[[], []] for _ in range(B)]
    held = np.zeros(B, np.int64)
    for step, counts in enumerate(([30, 1, 17], [1, 1, 1], [1, 1, 1], [3, 2, 1], [0, 5, 1], [1, 1, 1])):
        ptr = np.concatenate([[0], np.cumsum(counts)])
        n = int(ptr[-1])
        qkv = normal(gen, n, H + 2 * kv, dim, to=to)
        q, k, v = qkv[:, :H], qkv[:, H:H + kv], qkv[:, H + kv:]
        at = np.concatenate([np.arange(h, h + c) for h, c in zip(held, counts)])
        positions = torch.tensor(np.stack([np.full(n, step * 50), at]), dtype=torch.int32, device="cuda")
        turn = sn.HeadRotary(n, H, dim, n_kv_heads=kv, freqs=freqs, axes=axes, dtype=to)
        qt, kt = sn.head_rotary_forward(turn, q, k, positions, sn.head_rotary_workspace(turn), *w)
        for x, got, weight in ((q, qt, w[0]), (k, kt, w[1])):
            ref, factor = R.rotary(x, weight, positions, freqs, axes, False, True, 1e-6)
            R.check("turned", got, ref["y"], factor, dtype == "bfloat16")
        held += counts
        lengths = torch.from_numpy(held.astype(np.int32)).cuda()
        plan = sn.CacheRows(cache, ptr, 8, n_heads=H)
        ws = sn.cache_workspace(plan)
        sn.cache_write(plan, kt, v, table, lengths, ws)
        o = sn.cache_attend(plan, qt, table, lengths, ws)
        assert sn.read_status(ws) == sn.SN_OK
        for b in range(B):
            for i, x in enumerate((kt, v)):
                if counts[b]:
                    kept[b][i].append(R.held(x[ptr[b]:ptr[b + 1]], codes))
        ref, factor = R.attend(qt, [torch.cat(s[0]) for s in kept], [torch.cat(s[1]) for s in kept], ptr, held, plan.scale)
        R.check("o", o, ref["o"], factor, dtype == "bfloat16", 2.0 ** -16 if dtype == "bfloat16" else 0.0)


def test_history_as_states_of_the_cross_attention(sn):
    """Rows read back from the pages are the states of a cross attention of as many keys: both attentions agree."""
    import torch
    c = cache_case(sn, [1, 1, 1], [33, 120, 64], 2, 32, 16, "float32", "int8", 37, heads=4, causal=False)
    o = sn.cache_attend(c["plan"], c["q"], c["table"], c["lengths"], c["ws"])
    k, v = sn.cache_read(c["whole"], c["table"], c["lengths"], c["ws"])
    plan = sn.CrossAttention(c["row_ptr"], c["ptr"], 4, 2, 32)
    other = sn.cross_attention_forward(plan, c["q"], k, v, sn.cross_attention_workspace(plan))
    ref, factor = R.attend(c["q"], *kept_rows(c), c["row_ptr"], c["held"], plan.scale, False)
    R.check("pages", o, ref["o"], factor)
    R.check("states", other, ref["o"], factor + 2.0 ** -23)      # its states were rounded once more, to fp32

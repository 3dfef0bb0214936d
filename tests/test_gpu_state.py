"""GPU: the rotation of heads and the state cache against 64-bit references (state_ref.py states how the tolerances are
derived)."""
import numpy as np
import pytest

import state_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sn():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import schnet_cfconv_force_amd as sn
    sn.lib()
    return sn


def torch_type(name):
    import torch
    return {"float32": torch.float32, "bfloat16": torch.bfloat16}[name]


def normal(gen, *shape, to):
    import torch
    return torch.randn(shape, generator=gen, device="cuda").to(to)


# ------------------------------------------------------------------ rotation

def rotary_case(sn, rows, heads, kv, dim, sections, interleaved, norm, dtype, seed, far=1000, layout="plain", weights=True):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    to = torch_type(dtype)
    if layout == "plain":
        q, k = normal(gen, rows, heads, dim, to=to), normal(gen, rows, kv, dim, to=to)
    elif layout == "joined":        # one projection's rows
        qk = normal(gen, rows, heads + 2 * kv, dim, to=to)
        q, k = qk[:, :heads], qk[:, heads:heads + kv]
    else:                           # nothing aligned: rows begin at odd elements
        q = normal(gen, rows * heads * (dim + 1) + 1, to=to)[1:].view(rows, heads, dim + 1)[..., :dim]
        k = normal(gen, rows * kv * (dim + 3) + 1, to=to)[1:].view(rows, kv, dim + 3)[..., :dim]
    freqs, axes = (None, None) if not sections else sn.rotary_frequencies(sections)
    n_axes = max(len(sections), 1)
    positions = torch.randint(-far, far, (n_axes, rows), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    w = [normal(gen, dim, to=torch.float32) if norm and weights else None for _ in range(2)]
    g = [normal(gen, rows, n, dim, to=to) for n in (heads, kv)]
    plan = sn.HeadRotary(rows, heads, dim, n_kv_heads=kv, freqs=freqs, axes=axes, interleaved=interleaved, norm=norm, dtype=to)
    return plan, q, (k if kv else None), (positions if sections else None), w, g, freqs, axes


def rotary_check(sn, case, interleaved, norm, dtype, backward=True):
    import torch
    plan, q, k, positions, w, g, freqs, axes = case
    ws = sn.head_rotary_workspace(plan)
    out = sn.head_rotary_forward(plan, q, k, positions, ws, *w)
    grads = sn.head_rotary_backward(plan, q, k, positions, g[0], g[1] if k is not None else None, ws, *w) if backward else None
    torch.cuda.synchronize()
    assert sn.read_status(ws) == sn.SN_OK
    rounded = dtype == "bfloat16"
    worst = 0.0
    for i, x in enumerate((q, k)):
        if x is None:
            assert out[i] is None and (grads is None or (grads[i] is None and grads[2 + i] is None))
            continue
        ref, factor = R.rotary(x, w[i], positions, [] if freqs is None else freqs, [] if axes is None else axes, interleaved,
                               norm, 1e-6, g[i])
        worst = max(worst, R.check(f"y{i}", out[i], ref["y"], factor, rounded))
        if backward:
            worst = max(worst, R.check(f"dx{i}", grads[i], ref["dx"], factor, rounded))
            if norm:
                worst = max(worst, R.check(f"dw{i}", grads[2 + i], ref["dw"], factor))
            else:
                assert grads[2 + i] is None
    print(f"worst {worst:.3f} of the tolerance", flush=True)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("dim,sections", [(128, [16, 24, 24]), (32, [16]), (40, [5, 4, 3]), (40, [8, 12]), (16, [4, 4]), (1, []),
                                          (2, [1]), (7, [1, 2]), (80, [8, 8, 8, 8, 8]), (96, [16, 16]), (24, []), (127, [63]),
                                          (64, [1] * 8)], ids=str)
def test_rotary_head_sizes(sn, dim, sections, dtype, interleaved, norm):
    print(f"[rotary] {dim} {sections} {dtype} {interleaved} {norm}", flush=True)
    rotary_check(sn, rotary_case(sn, 37, 6, 2, dim, sections, interleaved, norm, dtype, dim), interleaved, norm, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,heads,kv", [(1, 1, 0), (1, 4, 4), (3, 1, 1), (2000, 8, 2), (4097, 3, 0), (70000, 2, 1), (0, 4, 4)])
def test_rotary_rows_and_heads(sn, rows, heads, kv, dtype):
    print(f"[rotary] rows {rows} heads {heads} {kv} {dtype}", flush=True)
    rotary_check(sn, rotary_case(sn, rows, heads, kv, 32, [8, 8], False, True, dtype, 3), False, True, dtype)


@pytest.mark.parametrize("layout", ["joined", "odd"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("dim", [32, 40, 128])
def test_rotary_strides(sn, dim, dtype, layout):
    print(f"[rotary] strides {dim} {dtype} {layout}", flush=True)
    rotary_check(sn, rotary_case(sn, 129, 6, 2, dim, [4, 8], False, True, dtype, 5, layout=layout), False, True, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_rotary_far_positions_and_no_weights(sn, dtype):
    """Positions to the type's ends: the angle is formed and reduced in fp64."""
    case = rotary_case(sn, 300, 4, 2, 64, [16, 16], False, True, dtype, 6, far=2 ** 31 - 1, weights=False)
    case[3][:, 0], case[3][:, 1] = -2 ** 31, 2 ** 31 - 1
    rotary_check(sn, case, False, True, dtype)


# ------------------------------------------------------------------ cache

def cache_case(sn, new, held, kv, dim, page, dtype, codes, seed, heads=None, spare=2, layout="plain", **attend):
    """A cache whose sequences hold `held` rows (written in one call) and a plan for their last `new` ones."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    to = torch_type(dtype)
    new, held = np.asarray(new, np.int64), np.asarray(held, np.int64)
    need = -(-held // page)
    max_pages = int(need.max()) + spare
    n_pages = int(need.sum()) + 3
    order = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((len(new), max_pages), -7, np.int32)
    for b, first in enumerate(np.cumsum(need) - need):
        table[b, :need[b]] = order[first:first + need[b]]
    cache = sn.StateCache(n_pages, page, kv, dim, dtype=to, codes=codes)
    ptr = np.concatenate([[0], np.cumsum(held)])
    spread = torch.exp(normal(gen, 2, kv, dim, to=torch.float32) * 0.3)
    n = int(ptr[-1])
    rows = [(normal(gen, n, kv, dim, to=torch.float32) * s).to(to) for s in spread]
    if layout == "odd":
        wide = [torch.zeros(n * kv * (dim + 1) + 1, dtype=to, device="cuda")[1:].view(n, kv, dim + 1)[..., :dim] for _ in range(2)]
        for w, r in zip(wide, rows):
            w.copy_(r)
        rows = wide
    elif layout == "joined":
        rows = list(torch.stack(rows, 1).unbind(1))
    table, lengths = torch.from_numpy(table).cuda(), torch.from_numpy(held.astype(np.int32)).cuda()
    whole = sn.CacheRows(cache, ptr, max_pages)
    ws = sn.cache_workspace(whole)
    sn.cache_write(whole, rows[0], rows[1], table, lengths, ws)
    assert sn.read_status(ws) == sn.SN_OK
    row_ptr = np.concatenate([[0], np.cumsum(new)])
    plan = sn.CacheRows(cache, row_ptr, max_pages, n_heads=heads, **attend)
    q = normal(gen, int(row_ptr[-1]), plan.n_heads, dim, to=to)
    return {"cache": cache, "plan": plan, "whole": whole, "ws": sn.cache_workspace(plan), "table": table, "lengths": lengths,
            "rows": rows, "ptr": ptr, "row_ptr": row_ptr, "held": held, "q": q, "codes": codes, "dtype": dtype}


def kept_rows(c):
    """Per sequence the held rows [length, Hkv, D] in float64, k and v."""
    return [[R.held(x[a:b], c["codes"]) if b > a else x[a:b].double().cpu() for a, b in zip(c["ptr"][:-1], c["ptr"][1:])]
            for x in c["rows"]]


def attend_check(sn, c, absent=None, status=0, plan=None):
    plan = plan or c["plan"]
    o, lse = sn.cache_attend(plan, c["q"], c["table"], c["lengths"], c["ws"], save=True)
    assert sn.read_status(c["ws"]) == status
    k, v = kept_rows(c)
    ref, factor = R.attend(c["q"], k, v, c["row_ptr"], c["held"], plan.scale, bool(plan.c.causal), plan.c.window, absent)
    rounded = c["dtype"] == "bfloat16"
    worst = R.check("o", o, ref["o"], factor, rounded, 2.0 ** -16 if rounded else 0.0)
    worst = max(worst, R.check("lse", lse, ref["lse"], 16 * R.U32))
    print(f"worst {worst:.3f} of the tolerance", flush=True)
    return o, lse


CODES = [None, "int8", "e4m3"]
TYPES = ["float32", "bfloat16"]


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,kv,layout", [(128, 16, 2, "plain"), (32, 32, 4, "joined"), (40, 16, 3, "odd"), (16, 64, 1, "joined"),
                                                (1, 16, 2, "plain"), (7, 128, 2, "plain"), (80, 16, 1, "odd"), (96, 1024, 2, "joined")])
def test_rows_written_are_read_back(sn, dim, page, kv, layout, dtype, codes):
    """Codes and scales equal the definition's to the bit; rows behind and between are left as they were."""
    import torch
    print(f"[cache] {dim} {page} {kv} {layout} {dtype} {codes}", flush=True)
    c = cache_case(sn, [1, 0, 5, 17, 2], [1, 3, 37, 17, 200], kv, dim, page, dtype, codes, dim + page, layout=layout)
    cache, page_at, at = c["cache"], *R.places(c["table"], page, c["ptr"], c["held"])
    touched = torch.zeros((cache.n_pages, page), dtype=torch.bool)
    touched[page_at, at] = True
    for x, pool, scales in zip(c["rows"], (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        got = pool.transpose(1, 2).float().cpu()
        if codes is None:
            assert torch.equal(got[page_at, at], x.float().cpu())
        else:
            y, scale = R.quantise(x, codes)
            assert np.array_equal(got[page_at, at].double().numpy(), y)
            assert np.array_equal(scales.transpose(1, 2).cpu().numpy()[page_at, at], scale)
            assert not bool(scales.transpose(1, 2).cpu()[~touched].any())
        assert not bool(got[~touched].any())
    k, v = sn.cache_read(c["plan"], c["table"], c["lengths"], c["ws"])
    assert sn.read_status(c["ws"]) == sn.SN_OK
    last = np.concatenate([np.arange(e - n, e) for e, n in zip(c["ptr"][1:], np.diff(c["row_ptr"]))]).astype(np.int64)
    for x, got in zip(c["rows"], (k, v)):
        want = R.held(x, codes)[last].to(torch.float32).to(x.dtype)      # the fp32 product of code and scale, rounded
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_codes_of_odd_rows(sn, dtype, codes):
    """Zeros, tiny rows, subnormals, the type's largest values, ties, infinities and NaN."""
    import torch
    to = torch_type(dtype)
    D = 32
    rows = [torch.zeros(D), torch.full((D,), 1e-38), torch.full((D,), 2.0 ** -100), torch.full((D,), 2.0 ** -101),
            torch.full((D,), torch.finfo(to).max), torch.arange(D) * 1.0 - 16, torch.linspace(-127, 127, D),
            torch.cat([torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -64.5]), torch.arange(24) + 0.5]),
            torch.cat([torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 432.0, 440.0]), torch.ones(24)]),
            torch.tensor([float("inf")] + [1.0] * (D - 1)), torch.tensor([1.0] * (D - 1) + [float("nan")]),
            torch.tensor([float("-inf"), float("nan")] * (D // 2))]
    x = torch.stack(rows).to(to)[:, None].cuda()
    n = len(rows)
    cache = sn.StateCache(2, 16, 1, D, dtype=to, codes=codes)
    plan = sn.CacheRows(cache, [0, n], 1)
    ws = sn.cache_workspace(plan)
    table, lengths = torch.tensor([[1]], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    sn.cache_write(plan, x, -x, table, lengths, ws)
    k, v = sn.cache_read(plan, table, lengths, ws)
    assert sn.read_status(ws) == sn.SN_OK
    for given, pool, scales, back in ((x, cache.k, cache.k_scale, k), (-x, cache.v, cache.v_scale, v)):
        y, scale = R.quantise(given[:, 0], codes)
        assert np.array_equal(pool[1, 0, :n].double().cpu().numpy(), y)
        assert np.array_equal(scales[1, 0, :n].cpu().numpy(), scale, equal_nan=True)
        want = torch.from_numpy(y * scale[:, None].astype(np.float64)).float().to(to)
        assert torch.equal(torch.isnan(back[:, 0].cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(back[:, 0].cpu(), 0.0), torch.nan_to_num(want, 0.0))


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,heads,kv,page", [(128, 8, 2, 16), (32, 4, 4, 32), (40, 6, 2, 16), (16, 8, 8, 64), (64, 16, 1, 16),
                                               (96, 40, 2, 16), (8, 3, 3, 256), (1, 1, 1, 16), (20, 34, 2, 16), (128, 1, 1, 16)])
def test_attend_head_layouts(sn, dim, heads, kv, page, dtype, codes):
    print(f"[attend] {dim} {heads}/{kv} {page} {dtype} {codes}", flush=True)
    c = cache_case(sn, [1, 1, 1, 1], [1, 300, 33, 64], kv, dim, page, dtype, codes, dim, heads=heads)
    attend_check(sn, c)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (True, 1000), (False, 0)])
def test_attend_masks(sn, causal, window, dtype, codes):
    """Several new rows, none, more rows than one tile; empty sequences for rows that see all."""
    print(f"[attend] causal {causal} window {window} {dtype} {codes}", flush=True)
    new = [3, 0, 7, 1, 20] if causal else [3, 2, 7, 0, 20]
    held = [3, 50, 130, 1, 261] if causal else [2, 0, 130, 5, 261]
    c = cache_case(sn, new, held, 2, 32, 16, dtype, codes, 11, heads=6, causal=causal, window=window)
    attend_check(sn, c)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,longest,heads,kv,dim", [(1, 20001, 4, 1, 32), (3, 5000, 8, 2, 128), (70, 700, 2, 2, 64)])
def test_attend_long_and_many(sn, batch, longest, heads, kv, dim, dtype, codes):
    print(f"[attend] {batch} x {longest} {heads}/{kv} x {dim} {dtype} {codes}", flush=True)
    held = np.random.default_rng(longest).integers(1, longest + 1, batch)
    held[-1] = longest
    c = cache_case(sn, np.ones(batch, np.int64), held, kv, dim, 16, dtype, codes, 12, heads=heads)
    attend_check(sn, c)


@pytest.mark.parametrize("dtype,codes", [("float32", None), ("bfloat16", "e4m3"), ("bfloat16", None)])
@pytest.mark.parametrize("batch,causal", [(70, True), (70, False), (300, False)])
def test_attend_sequences_that_share_blocks(sn, batch, causal, dtype, codes):
    """A table with room for far more rows than there are: all sequences' keys are one line that the blocks share."""
    print(f"[attend] shared {batch} {causal} {dtype} {codes}", flush=True)
    rng = np.random.default_rng(batch)
    held = rng.integers(1 if causal else 0, 900, batch)
    held[rng.integers(batch)] = 3000
    new = rng.integers(0, 3, batch)
    new = np.minimum(new, held) if causal else new
    c = cache_case(sn, new, held, 1, 32, 16, dtype, codes, 13, heads=3, spare=60000 // 16, causal=causal)
    attend_check(sn, c)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_many_rows_of_a_head(sn, dim, dtype, codes):
    """More rows than a tile of 16, few and many blocks of them (one and two tiles a block)."""
    print(f"[attend] rows {dim} {dtype} {codes}", flush=True)
    attend_check(sn, cache_case(sn, [5, 17, 0], [70, 33, 9], 2, dim, 16, dtype, codes, 14, heads=16))
    attend_check(sn, cache_case(sn, [5] * 70, list(range(5, 75)), 4, dim, 16, dtype, codes, 15, heads=32))

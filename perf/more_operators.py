"""The rotation and state cache operators and the cases they are measured on.

A norm and a rotation by positions on several axes of the query and key heads, forward and as a
training step; rows of keys and values written to a paged cache (as they are, or in 8 bits with a
scale for each row of a head) and read back; attention of a sequence's newest rows over its pages.
`own` selects between the plain form in torch operations and the library's kernels.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
_EPS = 1e-6
_TOP = {"int8": 127.0, "e4m3": 448.0}      # the largest code
_TINY = 2.0 ** -100                        # a row below this holds zeros


# ------------------------------------------------------------------ cases

def _rotary(name, mode, dtype, rows, heads, kv_heads, dim, sections, interleaved=False, norm=True):
    case = {"op": "rotary", "mode": mode, "dtype": dtype, "rows": rows, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "sections": sections, "interleaved": interleaved, "norm": norm}
    return dict(case, name=name) if name else case


def _store(name, dtype, codes, batch, new, held, kv_heads, dim, page, lengths):
    case = {"op": "store", "dtype": dtype, "codes": codes, "batch": batch, "new": new, "held": held,
            "kv_heads": kv_heads, "dim": dim, "page": page, "lengths": lengths}
    return dict(case, name=name) if name else case


def _attend(name, dtype, codes, batch, new, longest, heads, kv_heads, dim, page, lengths, causal=True, window=0):
    case = {"op": "attend", "dtype": dtype, "codes": codes, "batch": batch, "new": new, "longest": longest,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "lengths": lengths, "causal": causal,
            "window": window}
    return dict(case, name=name) if name else case


def listed():
    return [
        # the newest row of one chain, the bead features' own heads: the smallest call, all latency
        _rotary("rotate-step-f32", "forward", "float32", 1, 4, 4, 32, "16"),
        # fitting on the rows of 64 replicas of the 269-bead protein, positions (frame, residue)
        _rotary("rotate-train-replicas-f32", "train", "float32", 64 * 269, 4, 4, 32, "8+8"),
        # long sequences of wide rows whose keys are shared by four query heads, three axes
        _rotary("rotate-long-bf16", "forward", "bfloat16", 32768, 32, 8, 128, "16+24+24"),
        # fitting with an odd head size of which a part turns, adjacent pairs
        _rotary("rotate-train-odd-bf16", "train", "bfloat16", 7001, 6, 2, 40, "5+4+3", interleaved=True),
        # one new row of each of 64 sequences into 8 bits
        _store("store-step-e4m3", "bfloat16", "e4m3", 64, 1, 300, 8, 128, 16, 1),
        # the states of 64 chains in the framework's own 32-bit type, kept as they are
        _store("store-replicas-f32", "float32", "rows", 64, 271, 0, 4, 32, 32, 2),
        # whole histories of wide rows into 8 bits
        _store("store-history-int8", "bfloat16", "int8", 48, 4096, 100, 8, 128, 64, 3),
        # one query over the states of one 269-residue protein: the smallest call
        _attend("attend-one-chain-f32", "float32", "rows", 1, 1, 271, 4, 4, 32, 16, 4),
        # one new row of each of 64 replicas over short histories, 8-bit rows beside 32-bit queries
        _attend("attend-replicas-int8", "float32", "int8", 64, 1, 1076, 8, 8, 16, 32, 5, causal=False),
        # a few rows checked at once, an odd head size, heads shared by three, a window
        _attend("attend-draft-bf16", "bfloat16", "rows", 24, 5, 4099, 6, 2, 40, 64, 6, window=1500),
        # one new row per sequence over long histories with shared heads: all bytes of the cache
        _attend("attend-long-bf16", "bfloat16", "rows", 32, 1, 20000, 32, 8, 128, 16, 7),
        # the same histories in 8 bits
        _attend("attend-long-e4m3", "bfloat16", "e4m3", 32, 1, 20000, 32, 8, 128, 16, 7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["float32", "bfloat16"])
    codes = rng.choice(["rows", "int8", "e4m3"])
    lengths = rng.randrange(1 << 30)
    group = rng.choice([1, 1, 2, 3, 4, 8])
    kv_heads = _log_int(rng, 1, 8)
    dim = rng.choice([8, 16, 20, 24, 32, 32, 40, 64, 64, 80, 96, 128, 128])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    batch = _log_int(rng, 1, 64)
    kind = rng.random()
    if kind < 0.4:
        mode = rng.choice(["forward", "train"])
        rows = _log_int(rng, 1, 32768)
        while rows * kv_heads * (group + 1) * dim * (4 if dtype == "float32" else 2) * (2.5 if mode == "train" else 1) > 3.3e8:
            rows //= 2
        pairs = rng.randint(1, dim // 2)
        axes = min(pairs, rng.randint(1, 4))
        cuts = sorted(rng.sample(range(1, pairs), axes - 1)) if pairs > 1 else []
        sections = "+".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        return _rotary(None, mode, dtype, rows, kv_heads * group, kv_heads, dim, sections, rng.random() < 0.4,
                       rng.random() < 0.8)
    if kind < 0.6:
        new = 1 if rng.random() < 0.3 else _log_int(rng, 1, 4096)
        while batch * new * kv_heads * dim * (2 if dtype == "float32" else 1) > 48 * 2500 * 8 * 128:
            batch, new = max(1, batch // 2), max(1, new * 3 // 4)
        return _store(None, dtype, codes, batch, new, rng.choice([0, 1, 300]), kv_heads, dim, page, lengths)
    causal = rng.random() < 0.6
    new = 1 if rng.random() < 0.5 else rng.randint(2, 16)
    longest = max(new, _log_int(rng, 1, 20000))
    while batch > 1 and batch * longest * kv_heads * dim * (2 if dtype == "float32" else 1) > 32 * 12000 * 8 * 128:
        batch //= 2
    while batch > 1 and batch * longest * kv_heads * group * new > 2.5e7:
        batch //= 2
    window = _log_int(rng, 1, longest) if causal and rng.random() < 0.3 else 0
    return _attend(None, dtype, codes, batch, new, longest, kv_heads * group, kv_heads, dim, page, lengths, causal, window)


def _lengths(count, longest, least, key):
    """Row counts of the sequences: the longest and others down to a quarter of it, the case's own."""
    rng = np.random.default_rng([key, count, longest])
    n = rng.integers(max(least, longest // 4), longest + 1, count)
    n[rng.integers(count)] = longest
    return n


def _rows_of(case):
    """New rows and, with them, held rows of each sequence."""
    if case["op"] == "store":
        n = _lengths(case["batch"], case["new"], 1, case["lengths"])
        return n, n + _lengths(case["batch"], case["held"], 0, case["lengths"] + 1)
    n = np.full(case["batch"], case["new"], np.int64)
    held = _lengths(case["batch"], case["longest"], case["new"], case["lengths"])
    if case["batch"] > 2 and not case["causal"]:     # one sequence that holds nothing yet
        held[(held.argmax() + 1) % case["batch"]] = 0
    return n, held


def _sections(case):
    return [int(s) for s in case["sections"].split("+")]


def _frequencies(sections, base=10000.0):
    """One falling ladder over all pairs, cut into runs of one axis each."""
    pairs = sum(sections)
    return base ** (-np.arange(pairs) / pairs), np.repeat(np.arange(len(sections)), sections)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    device = "cuda"
    gen = torch.Generator(device=device).manual_seed(seed)
    dtype = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, to=dtype):
        return (torch.randn(shape, generator=gen, device=device) * scale + shift).to(to)

    if case["op"] == "rotary":
        rows, heads, kv_heads, dim = case["rows"], case["heads"], case["kv_heads"], case["dim"]
        # queries, keys and values side by side in a row, as one projection writes them
        qkv = normal(rows, heads + 2 * kv_heads, dim, scale=1.5)
        sections = _sections(case)
        place = torch.randint(0, 1 << 20, (1,), generator=gen, device=device)
        at = torch.arange(rows, device=device)
        positions = [place + at, at % 269, at // 269 - 3, 7 - at][:len(sections)]
        freqs, axes = _frequencies(sections)
        weights = [normal(dim, scale=0.2, shift=1.0, to=torch.float32) if case["norm"] else None for _ in range(2)]
        state = {
            "case": case,
            "q": qkv[:, :heads],
            "k": qkv[:, heads:heads + kv_heads],
            "positions": torch.stack(positions).to(torch.int32),
            "freqs": torch.from_numpy(freqs).to(device),
            "axes": torch.from_numpy(axes).to(device),
            "q_weight": weights[0],
            "k_weight": weights[1],
            "dq": normal(rows, heads, dim),
            "dk": normal(rows, kv_heads, dim),
        }
        if own:
            import schnet_cfconv_force_amd as sn
            state["plan"] = sn.HeadRotary(rows, heads, dim, n_kv_heads=kv_heads, freqs=freqs, axes=axes,
                                          interleaved=case["interleaved"], norm=case["norm"], eps=_EPS, dtype=dtype)
            state["ws"] = sn.head_rotary_workspace(state["plan"])
        return state

    new, held = _rows_of(case)
    batch, page, kv_heads, dim = case["batch"], case["page"], case["kv_heads"], case["dim"]
    pages = -(-held // page)
    max_pages = int(pages.max()) + 2                   # the table has room for rows to come
    n_pages = int(pages.sum()) + 3
    table = np.full((batch, max_pages), -1, np.int32)  # places that hold no page yet
    order = np.random.default_rng([seed, n_pages]).permutation(n_pages)
    for b, first in enumerate(np.cumsum(pages) - pages):
        table[b, :pages[b]] = order[first:first + pages[b]]
    row_ptr = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    state = {
        "case": case,
        "row_ptr": torch.from_numpy(row_ptr).to(device),
        "table": torch.from_numpy(table).to(device),
        "lengths": torch.from_numpy(held.astype(np.int32)).to(device),
    }
    # the rows of every sequence, each channel with a size of its own
    spread = torch.exp(normal(2, kv_heads, dim, scale=0.4, to=torch.float32))
    if case["op"] == "store":
        kv = (normal(int(row_ptr[-1]), 2, kv_heads, dim, to=torch.float32) * spread).to(dtype)
        state["k"], state["v"] = kv[:, 0], kv[:, 1]
    else:
        state["q"] = normal(int(row_ptr[-1]), case["heads"], dim)
        rows = int(held.sum())
        kv = [(normal(rows, kv_heads, dim, to=torch.float32) * s).to(dtype) for s in spread]
    if own:
        import schnet_cfconv_force_amd as sn
        cache = sn.StateCache(n_pages, page, kv_heads, dim, dtype=dtype, codes=None if case["codes"] == "rows" else case["codes"])
        state["cache"] = cache
        if case["op"] == "store":
            state["plan"] = sn.CacheRows(cache, row_ptr, max_pages)
        else:
            whole = sn.CacheRows(cache, np.concatenate([[0], np.cumsum(held)]), max_pages)
            sn.cache_write(whole, kv[0], kv[1], state["table"], state["lengths"], sn.cache_workspace(whole))
            state["plan"] = sn.CacheRows(cache, row_ptr, max_pages, n_heads=case["heads"], causal=case["causal"],
                                         window=case["window"])
        state["ws"] = sn.cache_workspace(state["plan"])
        return state
    kind = dtype if case["codes"] == "rows" else torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn
    pool = [torch.zeros((n_pages * page, kv_heads, dim), dtype=torch.float32, device=device).to(kind) for _ in range(2)]
    scales = [torch.zeros((n_pages * page, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    state.update(k_pool=pool[0], v_pool=pool[1], k_scale=scales[0], v_scale=scales[1])
    if case["op"] == "attend":
        slots = _slots(state["table"], page, held, held)
        _plain_write(state, slots, kv[0], kv[1])
    return state


def _slots(table, page, new, held):
    """Places in the pool of each sequence's last `new` rows (host counts)."""
    seq = np.repeat(np.arange(len(new)), new)
    at = np.arange(len(seq)) - np.repeat(np.cumsum(new) - new, new) + np.repeat(held - new, new)
    seq, at = (torch.from_numpy(t).to(table.device) for t in (seq, at))
    return table[seq, at // page].long() * page + at % page


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "store": _own_store, "attend": _own_attend}[op](state)
    return {"rotary": _plain_rotary, "store": _plain_store, "attend": _plain_attend}[op](state)


def _own_rotary(s):
    import schnet_cfconv_force_amd as sn
    weights = {"q_weight": s["q_weight"], "k_weight": s["k_weight"]}
    q, k = sn.head_rotary_forward(s["plan"], s["q"], s["k"], s["positions"], s["ws"], **weights)
    if s["case"]["mode"] == "forward":
        return {"q": q, "k": k}
    dq, dk, dqw, dkw = sn.head_rotary_backward(s["plan"], s["q"], s["k"], s["positions"], s["dq"], s["dk"], s["ws"], **weights)
    out = {"q": q, "k": k, "dq": dq, "dk": dk}
    return dict(out, dq_weight=dqw, dk_weight=dkw) if s["case"]["norm"] else out


def _own_store(s):
    import schnet_cfconv_force_amd as sn
    sn.cache_write(s["plan"], s["k"], s["v"], s["table"], s["lengths"], s["ws"])
    k, v = sn.cache_read(s["plan"], s["table"], s["lengths"], s["ws"])
    cache = s["cache"]
    out = {"k": k, "v": v, "k_pool": cache.k.transpose(1, 2), "v_pool": cache.v.transpose(1, 2)}
    if s["case"]["codes"] != "rows":
        out.update(k_scale=cache.k_scale.transpose(1, 2), v_scale=cache.v_scale.transpose(1, 2))
    return out


def _own_attend(s):
    import schnet_cfconv_force_amd as sn
    return sn.cache_attend(s["plan"], s["q"], s["table"], s["lengths"], s["ws"])


def _turn(t, cos, sin, interleaved):
    """The first 2 P elements of every head turned in pairs; the others as they are."""
    pairs = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = t[..., 0:2 * pairs:2], t[..., 1:2 * pairs:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = t[..., :pairs], t[..., pairs:2 * pairs]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, t[..., 2 * pairs:]], -1)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"][s["axes"]].double() * s["freqs"][:, None]     # far positions: 32 bits lose the angle
    cos, sin = torch.cos(angle).float().T, torch.sin(angle).float().T
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"]
        if c["norm"]:
            rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
            xh = x * rstd
        y = _turn(xh * w if c["norm"] else x, cos, sin, c["interleaved"])
        out[n] = y.to(s[n].dtype)
        if c["mode"] == "train":
            g = _turn(s["d" + n].float(), cos, -sin, c["interleaved"])
            if c["norm"]:
                out["d" + n + "_weight"] = (g * xh).sum((0, 1))
                g = g * w
                g = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
            out["d" + n] = g.to(s[n].dtype)
    return out


def _quantise(x, codes):
    """Codes and scales of rows [.., D] in 32 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, _TOP[codes])     # a tensor: quotients with a number are products with its inverse
    small, bad = amax < _TINY, ~torch.isfinite(amax)
    y = torch.where(small | bad, 0, x * (top / torch.where(small | bad, 1, amax)))
    scale = torch.where(bad, math.nan, torch.where(small, 0, amax / top))
    y = torch.round(y).to(torch.int8) if codes == "int8" else y.to(torch.float8_e4m3fn)
    return y, scale[..., 0]


def _plain_write(s, slots, k, v):
    for n, x in (("k", k), ("v", v)):
        if s["case"]["codes"] == "rows":
            s[n + "_pool"][slots] = x
        else:
            y, scale = _quantise(x.float(), s["case"]["codes"])
            s[n + "_pool"].view(torch.int8)[slots] = y.view(torch.int8)
            s[n + "_scale"][slots] = scale


def _plain_rows(s, n, slots):
    """Rows of the pool in 32 bits."""
    if s["case"]["codes"] == "rows":
        return s[n + "_pool"][slots].float()
    kind = s[n + "_pool"].dtype
    return s[n + "_pool"].view(torch.int8)[slots].view(kind).float() * s[n + "_scale"][slots][..., None]


def _plain_store(s):
    c = s["case"]
    new = (s["row_ptr"][1:] - s["row_ptr"][:-1]).long()
    rows = torch.arange(s["k"].shape[0], device=new.device)
    seq = torch.searchsorted(s["row_ptr"][1:].long(), rows, right=True)
    at = rows - s["row_ptr"].long()[seq] + (s["lengths"].long() - new)[seq]
    slots = s["table"][seq, at // c["page"]].long() * c["page"] + at % c["page"]
    _plain_write(s, slots, s["k"], s["v"])
    out = {n: _plain_rows(s, n, slots).to(s["k"].dtype) for n in ("k", "v")}
    shape = (-1, c["page"], c["kv_heads"])
    out.update(k_pool=s["k_pool"].view(*shape, c["dim"]), v_pool=s["v_pool"].view(*shape, c["dim"]))
    if c["codes"] != "rows":
        out.update(k_scale=s["k_scale"].view(shape), v_scale=s["v_scale"].view(shape))
    return out


def _plain_attend(s):
    c = s["case"]
    batch, new, kv_heads, dim = c["batch"], c["new"], c["kv_heads"], c["dim"]
    group, longest = c["heads"] // kv_heads, int(_rows_of(c)[1].max())
    at = torch.arange(longest, device="cuda")
    slots = s["table"][:, at // c["page"]].long().clamp(min=0) * c["page"] + at % c["page"]
    inside = at < s["lengths"][:, None]

    def keys(n):        # [B, Hkv, L, D], absent rows zero
        return torch.where(inside[:, :, None, None], _plain_rows(s, n, slots), 0).permute(0, 2, 1, 3).contiguous()

    q = s["q"].float().view(batch, new, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv_heads, group * new, dim)
    score = torch.matmul(q, keys("k").transpose(2, 3).contiguous()) * (1 / math.sqrt(dim))
    seen = inside[:, None].expand(batch, new, longest)
    if c["causal"]:
        own_at = s["lengths"][:, None] - new + torch.arange(new, device="cuda")
        seen = seen & (at <= own_at[:, :, None])
        if c["window"]:
            seen = seen & (at > own_at[:, :, None] - c["window"])
    score = torch.where(seen[:, None, None], score.view(batch, kv_heads, group, new, longest), -math.inf)
    top = score.amax(4, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0))
    total = p.sum(4, keepdim=True)
    p = (p / torch.where(total > 0, total, 1)).view(batch, kv_heads, group * new, longest)
    o = torch.matmul(p, keys("v"))
    return o.view(batch, kv_heads, group, new, dim).permute(0, 3, 1, 2, 4).reshape(batch * new, c["heads"], dim).to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = _TYPES[case["dtype"]].itemsize
    if case["op"] == "rotary":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        train = case["mode"] == "train"
        # forward x, y; a training step also dy, dx (x read once)
        return {"bytes": n * size * (4 if train else 2) + 4 * case["rows"] * len(_sections(case)), "flops": n * (20 if train else 8)}
    new, held = _rows_of(case)
    head_row = case["dim"] * (size if case["codes"] == "rows" else 1) + (0 if case["codes"] == "rows" else 4)
    if case["op"] == "store":       # the rows in, the rows held, the rows out
        n = 2 * int(new.sum()) * case["kv_heads"]
        return {"bytes": n * (2 * case["dim"] * size + head_row), "flops": 4 * n * case["dim"]}
    seen = np.minimum(held, case["window"] + case["new"] - 1) if case["window"] else held
    q = 2 * case["batch"] * case["new"] * case["heads"] * case["dim"]
    return {"bytes": 2 * int(seen.sum()) * case["kv_heads"] * head_row + q * size,
            "flops": 4 * int(seen.sum()) * case["new"] * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    global own
    before, own = own, False        # the inputs alone, without the library's plans
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"rotary": _exact_rotary, "store": _exact_store, "attend": _exact_attend}[case["op"]](case, s)


def _exact_rotary(case, s):
    sections = _sections(case)
    pairs, dim = sum(sections), case["dim"]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    out = {}
    for n in ("q", "k"):
        x = s[n].double()
        y, dx = torch.empty_like(x), torch.empty_like(x)
        w = s[n + "_weight"].double() if case["norm"] else torch.ones(dim, dtype=torch.float64, device=x.device)
        g = s["d" + n].double()
        z = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / dim + _EPS) if case["norm"] else x
        y[:], dx[:] = z * w, g
        for j in range(pairs):
            a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + pairs)
            turn = s["positions"][axis[j]].double()[:, None] * 10000.0 ** (-j / pairs)
            c, d = torch.cos(turn), torch.sin(turn)
            y[..., a], y[..., b] = z[..., a] * w[a] * c - z[..., b] * w[b] * d, z[..., a] * w[a] * d + z[..., b] * w[b] * c
            dx[..., a], dx[..., b] = g[..., a] * c + g[..., b] * d, g[..., b] * c - g[..., a] * d
        out[n] = y
        if case["mode"] == "train":
            if case["norm"]:
                out["d" + n + "_weight"] = (dx * z).sum(0).sum(0)
                h = dx * w
                sd = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / dim + _EPS)
                dx = h / sd - x * (h * x).sum(-1, keepdim=True) / (dim * sd ** 3)
            out["d" + n] = dx
    return out


def _exact_codes(x, codes):
    """The codes' values and the scales: quotients and products are rounded to 32 bits where the definition has them."""
    to32 = lambda t: t.float().double()     # noqa: E731
    x, top = x.double(), _TOP[codes]
    amax = x.abs().amax(-1, keepdim=True)
    live = (amax >= _TINY) & torch.isfinite(amax)
    y = to32(x * to32(top / torch.where(live, amax, 1.0)))
    if codes == "int8":
        y = torch.round(y)
    else:       # three bits behind the leading one; the smallest exponent is -6
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
        y = (torch.round(y / step) * step).clamp(-448, 448)
    return torch.where(live, y, 0.0), torch.where(live, to32(amax / top), 0.0)[..., 0]


def _exact_store(case, s):
    new, held = _rows_of(case)
    page, table = case["page"], s["table"].cpu().numpy()
    out = {}
    first = np.cumsum(new) - new
    places = np.concatenate([table[b, np.arange(h - n, h) // page].astype(np.int64) * page + np.arange(h - n, h) % page
                             for b, (n, h) in enumerate(zip(new, held))]) if len(first) else np.zeros(0, np.int64)
    places = torch.from_numpy(places).to(s["k"].device)
    pools, scales = {}, {}
    for n in ("k", "v"):
        pool = torch.zeros(s[n + "_pool"].shape, dtype=torch.float64, device=places.device)
        if case["codes"] == "rows":
            out[n], pool[places] = s[n].double(), s[n].double()
        else:
            y, scale = _exact_codes(s[n], case["codes"])
            out[n], pool[places] = y * scale[..., None], y
            full = torch.zeros(pool.shape[:2], dtype=torch.float64, device=places.device)
            full[places] = scale
            scales[n + "_scale"] = full.view(-1, page, case["kv_heads"])
        pools[n + "_pool"] = pool.view(-1, page, case["kv_heads"], case["dim"])
    return {**out, **pools, **scales}


def _exact_attend(case, s):
    new, held = _rows_of(case)
    page, group = case["page"], case["heads"] // case["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, length in enumerate(held.tolist()):
        if length == 0:
            continue
        at = torch.arange(length, device=o.device)
        slot = s["table"][b].long()[at // page] * page + at % page
        rows = slice(b * case["new"], (b + 1) * case["new"])
        hidden = torch.zeros((case["new"], length), dtype=torch.bool, device=o.device)
        if case["causal"]:
            ahead = at[None] - (length - case["new"] + torch.arange(case["new"], device=o.device))[:, None]
            hidden = ahead > 0
            if case["window"]:
                hidden = hidden | (ahead <= -case["window"])
        for h in range(case["kv_heads"]):
            k, v = ((s[n + "_pool"].view(torch.int8) if case["codes"] == "e4m3" else s[n + "_pool"])[slot, h] for n in ("k", "v"))
            if case["codes"] == "e4m3":
                k, v = k.view(torch.float8_e4m3fn).float(), v.view(torch.float8_e4m3fn).float()
            k, v = k.double(), v.double()
            if case["codes"] != "rows":
                k, v = k * s["k_scale"][slot, h].double()[:, None], v * s["v_scale"][slot, h].double()[:, None]
            for g in range(h * group, (h + 1) * group):
                a = (s["q"][rows, g].double() @ k.T.contiguous() / math.sqrt(case["dim"])).masked_fill(hidden, -math.inf)
                o[rows, g] = torch.softmax(a, 1) @ v
    return o

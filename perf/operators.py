"""The context operators and the cases they are measured on.

Cross attention of bead rows to an encoder's states of another length, with a learned relative
position bias by buckets, and a group norm with an activation over the rows of a replica; each
forward, and as a training step (forward and backward).  `own` selects between the plain form in
torch operations and the library's kernels.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
_LN2 = math.log(2.0)


# ------------------------------------------------------------------ cases

def _attention(name, mode, dtype, batch, lq, lk, heads, kv_heads, dim, bias=True, keep=True, ragged=True, lengths=0):
    case = {"op": "attention", "mode": mode, "dtype": dtype, "batch": batch, "lq": lq, "lk": lk, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "bias": bias, "keep": keep, "ragged": ragged, "lengths": lengths}
    return dict(case, name=name) if name else case


def _norm(name, mode, dtype, batch, rows, channels, groups, act, ragged=True, lengths=0):
    case = {"op": "norm", "mode": mode, "dtype": dtype, "batch": batch, "rows": rows, "channels": channels,
            "groups": groups, "act": act, "ragged": ragged, "lengths": lengths}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one pooled query over the states of one 269-residue protein: the smallest call, all latency
        _attention("pool-one-chain-f32", "forward", "float32", 1, 1, 269, 4, 4, 32, ragged=False),
        # one new query per sequence over long cached states with shared heads: all bytes of K and V
        _attention("pool-long-bf16", "forward", "bfloat16", 32, 1, 16384, 32, 8, 128, bias=False, lengths=1),
        # the bead features of 64 replicas of the 269-bead protein over the states of their sequence
        _attention("replicas-f32", "forward", "float32", 64, 269, 271, 4, 4, 32, lengths=2),
        # the 15,668-particle system as one segment over 1,000 states: long queries, narrow heads
        _attention("box-f32", "forward", "float32", 1, 15668, 1000, 8, 8, 16, ragged=False),
        # long sequences on both sides, wide heads, heads shared by four
        _attention("long-bf16", "forward", "bfloat16", 2, 4096, 4096, 16, 4, 128, ragged=False),
        # fitting the block on 64 replicas in the framework's own 32-bit type
        _attention("train-replicas-f32", "train", "float32", 64, 269, 271, 4, 4, 32, lengths=3),
        # fitting on chains of every length, an odd head size, heads shared by three
        _attention("train-odd-bf16", "train", "bfloat16", 24, 701, 517, 6, 2, 40, lengths=4),
        # a wide training step on long sequences
        _attention("train-long-bf16", "train", "bfloat16", 2, 2048, 2048, 16, 16, 64, lengths=5),
        # the bead features of one protein: a small call
        _norm("norm-chain-f32", "forward", "float32", 1, 269, 128, 8, "ssp", ragged=False),
        # one segment of 15,668 particles: one replica across the whole card
        _norm("norm-box-f32", "forward", "float32", 1, 15668, 128, 8, "ssp", ragged=False),
        # fitting on 64 replicas
        _norm("norm-train-replicas-f32", "train", "float32", 64, 269, 128, 8, "ssp", lengths=6),
        # long segments of wide rows, as an encoder's own norms meet them
        _norm("norm-train-wide-bf16", "train", "bfloat16", 8, 16384, 512, 32, "silu", lengths=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["float32", "bfloat16"])
    lengths = rng.randrange(1 << 30)
    ragged = rng.random() < 0.7
    if rng.random() < 0.35:
        mode = rng.choice(["forward", "train"])
        per = _log_int(rng, 1, 32)                 # channels of a group
        groups = _log_int(rng, 1, 32)
        channels = min(per * groups, 512) // groups * groups
        rows = _log_int(rng, 1, 16384)
        batch = _log_int(rng, 1, 64)
        while batch * rows * channels > 8 * 16384 * 512 // 2:
            batch = max(1, batch // 2)
            rows = rows if batch > 1 else rows // 2
        return _norm(None, mode, dtype, batch, rows, channels, groups, rng.choice(["none", "ssp", "silu"]), ragged, lengths)
    mode = rng.choice(["forward", "forward", "train"])
    few = mode == "forward" and rng.random() < 0.4
    lq = _log_int(rng, 1, 16) if few else _log_int(rng, 17, 4096)
    lk = _log_int(rng, 1, 16384 if few else 4096)
    group = rng.choice([1, 1, 2, 3, 4, 8])
    kv_heads = _log_int(rng, 1, max(1, 16 // group))
    dim = rng.choice([8, 16, 20, 24, 32, 32, 40, 64, 64, 80, 96, 128, 128])
    batch = _log_int(rng, 1, 64)
    heads = kv_heads * group
    # no more work or scores than the largest listed cases have
    while batch > 1 and (batch * heads * lq * lk > 1.2e8 or batch * lk * kv_heads * dim > 1.2e8):
        batch //= 2
    while heads * lq * lk > 1.2e8:
        lq, lk = max(1, lq // 2), max(1, lk // 2)
    return _attention(None, mode, dtype, batch, lq, lk, heads, kv_heads, dim, rng.random() < 0.7, rng.random() < 0.5,
                      ragged, lengths)


def _lengths(count, longest, ragged, key):
    """Row counts of the segments: the longest and others down to a quarter of it, the case's own."""
    if not ragged or count == 1:
        return np.full(count, longest, np.int64)
    rng = np.random.default_rng([key, count, longest])
    n = rng.integers(max(1, longest // 4), longest + 1, count)
    n[rng.integers(count)] = longest
    return n


def _pointers(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _attention_lengths(case):
    nq = _lengths(case["batch"], case["lq"], case["ragged"], case["lengths"])
    nk = _lengths(case["batch"], case["lk"], case["ragged"], case["lengths"] + 1)
    return nq, nk


# Buckets of the relative position: one per offset near zero, then wider ones by the logarithm, the
# outermost open-ended; bucket(rel) = number of thresholds <= rel.
def _thresholds(buckets=32, far=128):
    half, near = buckets // 2, buckets // 4
    wide = [near * (far / near) ** (j / (half - near)) for j in range(half - near)]
    steps = list(range(1, near)) + [int(math.ceil(w - 1e-9)) for w in wide]     # smallest distance of each bucket
    return [-(s - 1) for s in reversed(steps)] + [1] + [s + 1 for s in steps]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    device = "cuda"
    gen = torch.Generator(device=device).manual_seed(seed)
    dtype = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, to=dtype):
        return (torch.randn(shape, generator=gen, device=device) * scale + shift).to(to)

    if case["op"] == "norm":
        ptr = _pointers(_lengths(case["batch"], case["rows"], case["ragged"], case["lengths"]))
        rows, channels = int(ptr[-1]), case["channels"]
        state = {
            "case": case,
            "ptr": torch.from_numpy(ptr).to(device),
            "x": (normal(rows, channels, to=torch.float32) * 1.5 + normal(channels, to=torch.float32)).to(dtype),
            "gamma": normal(channels, scale=0.2, shift=1.0, to=torch.float32),
            "beta": normal(channels, scale=0.2, to=torch.float32),
            "dy": normal(rows, channels),
        }
        if own:
            import schnet_cfconv_force_amd as sn
            state["plan"] = sn.GroupNorm(ptr, channels, case["groups"], activation=case["act"], dtype=dtype)
            state["ws"] = sn.group_norm_workspace(state["plan"])
        return state

    nq, nk = _attention_lengths(case)
    q_ptr, k_ptr = _pointers(nq), _pointers(nk)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    # keys and values lie side by side in a row, as one projection of the states writes them
    kv = normal(int(k_ptr[-1]), 2, kv_heads, dim)
    keep = torch.rand(int(k_ptr[-1]), generator=gen, device=device) < 0.9
    # bead i of a chain against state j of the same chain's sequence; a one-row query pools from the middle
    q_pos = np.concatenate([np.arange(n) if n > 16 else np.arange(n) + m // 2 for n, m in zip(nq, nk)])
    k_pos = np.concatenate([np.arange(m) - 1 for m in nk])
    state = {
        "case": case,
        "q_ptr": torch.from_numpy(q_ptr).to(device),
        "k_ptr": torch.from_numpy(k_ptr).to(device),
        "q": normal(int(q_ptr[-1]), heads, dim),
        "k": kv[:, 0],
        "v": kv[:, 1],
        "do": normal(int(q_ptr[-1]), heads, dim),
        "keep": keep if case["keep"] else None,
        "bias": normal(heads, 32, scale=0.5, to=torch.float32) if case["bias"] else None,
        "q_pos": torch.from_numpy(q_pos.astype(np.int32)).to(device) if case["bias"] else None,
        "k_pos": torch.from_numpy(k_pos.astype(np.int32)).to(device) if case["bias"] else None,
        "thresholds": torch.tensor(_thresholds(), dtype=torch.int32, device=device),
    }
    if case["batch"] > 2 and case["keep"]:      # one segment whose states are all padding
        state["keep"][int(k_ptr[1]):int(k_ptr[2])] = False
    if own:
        import schnet_cfconv_force_amd as sn
        thresholds = sn.relative_thresholds(32, 128) if case["bias"] else None
        state["plan"] = sn.CrossAttention(q_ptr, k_ptr, heads, kv_heads, dim, dtype=dtype, thresholds=thresholds)
        state["ws"] = sn.cross_attention_workspace(state["plan"])
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    return _own_attention(state) if own else _plain_attention(state)


def _own_norm(s):
    import schnet_cfconv_force_amd as sn
    if s["case"]["mode"] == "forward":
        return sn.group_norm_forward(s["plan"], s["x"], s["gamma"], s["beta"], s["ws"])
    y, saved = sn.group_norm_forward(s["plan"], s["x"], s["gamma"], s["beta"], s["ws"], save=True)
    dx, dgamma, dbeta = sn.group_norm_backward(s["plan"], s["x"], s["gamma"], s["beta"], saved, s["dy"], s["ws"])
    return {"y": y, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _own_attention(s):
    import schnet_cfconv_force_amd as sn
    where = {"bias": s["bias"], "q_pos": s["q_pos"], "k_pos": s["k_pos"], "keep": s["keep"]}
    if s["case"]["mode"] == "forward":
        return sn.cross_attention_forward(s["plan"], s["q"], s["k"], s["v"], s["ws"], **where)
    o, saved = sn.cross_attention_forward(s["plan"], s["q"], s["k"], s["v"], s["ws"], save=True, **where)
    dq, dk, dv, dbias = sn.cross_attention_backward(s["plan"], s["q"], s["k"], s["v"], saved, s["do"], s["ws"], **where)
    out = {"o": o, "dq": dq, "dk": dk, "dv": dv}
    return dict(out, dbias=dbias) if dbias is not None else out


def _padded(ptr, longest, total):
    """Row index and validity [B, longest] of ragged rows, and each row's place in the padded layout."""
    at = torch.arange(longest, device=ptr.device)
    start, end = ptr[:-1, None].long(), ptr[1:, None].long()
    rows = torch.arange(total, device=ptr.device)
    seg = torch.searchsorted(ptr[1:].long(), rows, right=True)
    return (start + at).clamp(max=total - 1), start + at < end, seg * longest + rows - ptr.long()[seg]


def _activate(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "ssp":
        return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())) - _LN2
    return z


def _activate_grad(z, act):
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig)) if act == "silu" else sig if act == "ssp" else torch.ones_like(z)


def _plain_norm(s):
    c = s["case"]
    rows, channels = s["x"].shape
    idx, valid, place = _padded(s["ptr"], c["rows"], rows)
    shape = (c["batch"], c["rows"], c["groups"], channels // c["groups"])
    inside = valid[:, :, None, None]
    x = s["x"].float()[idx].view(shape)
    count = (valid.sum(1) * shape[3]).view(-1, 1, 1, 1).float()
    mean = torch.where(inside, x, 0).sum((1, 3), keepdim=True) / count
    centred = torch.where(inside, x - mean, 0)
    rstd = 1 / torch.sqrt((centred * centred).sum((1, 3), keepdim=True) / count + 1e-5)
    xh = centred * rstd
    gamma = s["gamma"].view(shape[2:])
    z = xh * gamma + s["beta"].view(shape[2:])

    def ragged(t):
        return t.reshape(-1, channels)[place].to(s["x"].dtype)

    y = ragged(_activate(z, c["act"]))
    if c["mode"] == "forward":
        return y
    dz = torch.where(inside, s["dy"].float()[idx].view(shape) * _activate_grad(z, c["act"]), 0)
    dxh = dz * gamma
    m1 = dxh.sum((1, 3), keepdim=True) / count
    m2 = (dxh * xh).sum((1, 3), keepdim=True) / count
    return {"y": y, "dx": ragged(rstd * (dxh - m1 - xh * m2)), "dgamma": (dz * xh).sum((0, 1)).view(-1),
            "dbeta": dz.sum((0, 1)).view(-1)}


def _plain_attention(s):
    c = s["case"]
    batch, kv_heads, dim, lq, lk = c["batch"], c["kv_heads"], c["dim"], c["lq"], c["lk"]
    group, dtype = c["heads"] // kv_heads, s["q"].dtype
    iq, okq, q_place = _padded(s["q_ptr"], lq, s["q"].shape[0])
    ik, okk, k_place = _padded(s["k_ptr"], lk, s["k"].shape[0])
    if s["keep"] is not None:
        okk = okk & s["keep"][ik]

    def queries(t):     # [B, Hkv, G Lq, D]: the heads that share keys and values lie together
        return t.float()[iq].view(batch, lq, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv_heads, group * lq, dim)

    def keys(t):        # [B, Hkv, Lk, D], absent rows zero
        return torch.where(okk[:, :, None, None], t.float()[ik], 0).permute(0, 2, 1, 3).contiguous()

    def from_queries(t):
        return t.view(batch, kv_heads, group, lq, dim).permute(0, 3, 1, 2, 4).reshape(-1, kv_heads * group, dim)[q_place].to(dtype)

    def from_keys(t):
        return t.permute(0, 2, 1, 3).reshape(-1, kv_heads, dim)[k_place].to(dtype)

    q, k, v = queries(s["q"]), keys(s["k"]), keys(s["v"])
    scale = 1 / math.sqrt(dim)
    score = (torch.matmul(q, k.transpose(2, 3).contiguous()) * scale).view(batch, kv_heads, group, lq, lk)
    if s["bias"] is not None:
        rel = s["k_pos"][ik][:, None, :] - s["q_pos"][iq][:, :, None]
        bucket = torch.searchsorted(s["thresholds"], rel, right=True)
        score += s["bias"][:, bucket].view(kv_heads, group, batch, lq, lk).permute(2, 0, 1, 3, 4)
    both = okq[:, None, None, :, None] & okk[:, None, None, None, :]
    score = torch.where(both, score, -math.inf)
    top = score.amax(4, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0))
    total = p.sum(4, keepdim=True)
    p = (p / torch.where(total > 0, total, 1)).view(batch, kv_heads, group * lq, lk)
    o = from_queries(torch.matmul(p, v))
    if c["mode"] == "forward":
        return o
    do = queries(s["do"])
    dp = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = p * (dp - (p * dp).sum(3, keepdim=True))
    out = {"o": o, "dq": from_queries(torch.matmul(ds, k) * scale),
           "dk": from_keys(torch.matmul(ds.transpose(2, 3).contiguous(), q) * scale),
           "dv": from_keys(torch.matmul(p.transpose(2, 3).contiguous(), do))}
    if s["bias"] is not None:
        rows = ds.view(batch, kv_heads * group, lq, lk)
        sums = torch.zeros((batch, kv_heads * group, lq, 32), device=ds.device)
        sums.scatter_add_(3, bucket[:, None].expand(rows.shape), rows)
        out["dbias"] = sums.sum((0, 2))
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = _TYPES[case["dtype"]].itemsize
    train = case["mode"] == "train"
    if case["op"] == "norm":
        n = int(_lengths(case["batch"], case["rows"], case["ragged"], case["lengths"]).sum()) * case["channels"]
        # forward x, y; a training step also dy, dx (x read once)
        return {"bytes": n * size * (4 if train else 2), "flops": n * (30 if train else 12)}
    nq, nk = _attention_lengths(case)
    pairs = int((nq * nk).sum()) * case["heads"]
    rows = int(nq.sum()) * case["heads"] * case["dim"]
    states = 2 * int(nk.sum()) * case["kv_heads"] * case["dim"]
    # forward q, k, v, o; a training step also do, dq, dk, dv.  Products: q k, p v; and do v, p do, ds k, ds q
    return {"bytes": size * ((4 if train else 2) * rows + (2 if train else 1) * states),
            "flops": (12 if train else 4) * case["dim"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    global own
    before, own = own, False        # the inputs alone, without the library's plans
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_attention(case, s)


def _exact_norm(case, s):
    ptr = s["ptr"].tolist()
    x, dy = s["x"].double(), s["dy"].double()
    rows, channels = x.shape
    width = channels // case["groups"]
    gamma, beta = s["gamma"].double(), s["beta"].double()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(beta)
    for a, b in zip(ptr[:-1], ptr[1:]):
        part = x[a:b].reshape(b - a, case["groups"], width)
        mean = part.mean((0, 2))[None, :, None]
        var = ((part - mean) ** 2).mean((0, 2))[None, :, None]
        sd = torch.sqrt(var + 1e-5)
        xh = ((part - mean) / sd).reshape(b - a, channels)
        z = xh * gamma + beta
        if case["act"] == "none":
            f, slope = z, torch.ones_like(z)
        elif case["act"] == "ssp":
            f = torch.logaddexp(z, torch.zeros_like(z)) - math.log(2)
            slope = torch.sigmoid(z)
        else:
            f = z * torch.sigmoid(z)
            slope = torch.sigmoid(z) + f * (1 - torch.sigmoid(z))
        y[a:b] = f
        g = dy[a:b] * slope
        dgamma += (g * xh).sum(0)
        dbeta += g.sum(0)
        h = (g * gamma).reshape(b - a, case["groups"], width)
        e = xh.reshape(h.shape)
        d = (h - h.mean((0, 2))[None, :, None] - e * (h * e).mean((0, 2))[None, :, None]) / sd
        dx[a:b] = d.reshape(b - a, channels)
    return y if case["mode"] == "forward" else {"y": y, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _exact_attention(case, s):
    q_at, k_at = s["q_ptr"].tolist(), s["k_ptr"].tolist()
    q, k, v, g = (s[n].double() for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    group, train = case["heads"] // case["kv_heads"], case["mode"] == "train"
    edges = s["thresholds"]
    dbias = torch.zeros((case["heads"], len(edges) + 1), dtype=torch.float64, device=q.device)
    for b in range(case["batch"]):
        rows = slice(q_at[b], q_at[b + 1])
        cols = torch.arange(k_at[b], k_at[b + 1], device=q.device)
        if s["keep"] is not None:
            cols = cols[s["keep"][cols]]
        if cols.numel() == 0 or rows.start == rows.stop:
            continue
        if s["bias"] is not None:
            bucket = torch.bucketize(s["k_pos"][cols][None, :] - s["q_pos"][rows][:, None], edges, right=True)
        for h in range(case["heads"]):
            kh, vh, qh = k[cols, h // group], v[cols, h // group], q[rows, h]
            a = qh @ kh.T.contiguous() / math.sqrt(case["dim"])
            if s["bias"] is not None:
                a = a + s["bias"][h].double()[bucket]
            p = torch.softmax(a, 1)
            o[rows, h] = p @ vh
            if not train:
                continue
            gh = g[rows, h]
            dp = gh @ vh.T.contiguous()
            ds = p * (dp - (gh * o[rows, h]).sum(1, keepdim=True))
            dq[rows, h] = ds @ kh / math.sqrt(case["dim"])
            dk[cols, h // group] += ds.T.contiguous() @ qh / math.sqrt(case["dim"])
            dv[cols, h // group] += p.T.contiguous() @ gh
            if s["bias"] is not None:
                dbias[h] += torch.bincount(bucket.reshape(-1), ds.reshape(-1), minlength=len(edges) + 1)
    if not train:
        return o
    out = {"o": o, "dq": dq, "dk": dk, "dv": dv}
    return dict(out, dbias=dbias) if s["bias"] is not None else out

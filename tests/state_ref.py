"""64-bit references of the rotation of heads and of the state cache, with the magnitudes that bound their rounding
errors.

Tolerances.  u = 2^-24 is half a unit of fp32.  Rotation: a head's mean square is a sum of at most 128 squares joined
in a tree or in runs of 16, and rstd, the two products, the angle (fp32 of the part of a turn that is left: 2^-25 of a
turn, 3 u of angle), sine and cosine (2 u each), the turn's products and its sum add a few u each: 48 u of |z_a| + |z_b|
covers them.  Positions near the type's ends move the angle by 2^31 2^-52, 8 u more: 64 u.  Gradients
carry the same errors twice (of g and of xh).  Codes are exact.  Attention: an inner product of at most 128 terms, an exponential
and a normalisation: 128 u of the sum of the magnitudes while the scores stay within about 8; larger ones amplify an
error of s in exp(s), so the factor grows with max |s| / 8.  Every output is a sum; its error is taken relative to the
same sum over magnitudes.  A bf16 output adds its rounding, 2^-8 of its value, and attention the 16 bits of the weights,
2^-16 of the magnitudes.
"""
import math

import numpy as np
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8
TOP = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ rotation

def pairs_of(n_pairs, interleaved):
    j = np.arange(n_pairs)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + n_pairs)


def rotary(x, w, positions, freqs, axes, interleaved, norm, eps, dy=None):
    """dict name -> (value, magnitudes) in float64 on the CPU: y, and with dy also dx and (with a norm) dw."""
    x = x.detach().double().cpu()
    D = x.shape[-1]
    w = torch.ones(D, dtype=torch.float64) if w is None else w.detach().double().cpu()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if norm else torch.ones(())
    xh = x * rstd
    z = xh * w if norm else xh
    pa, pb = pairs_of(len(freqs), interleaved)
    pos = np.zeros((1, x.shape[0]), np.int64) if positions is None else positions.cpu().numpy().astype(np.int64)
    angle = torch.from_numpy(pos[np.asarray(axes, np.int64)].T * np.asarray(freqs)[None]) if len(freqs) else None

    def turn(t, sign):
        v, m = t.clone(), t.abs()
        if len(freqs):
            c, s = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
            a, b = t[..., pa], t[..., pb]
            v[..., pa], v[..., pb] = a * c - b * s, b * c + a * s
            m[..., pa] = m[..., pb] = a.abs() + b.abs()
        return v, m

    out = {"y": turn(z, 1.0)}
    if dy is not None:
        g, gm = turn(dy.detach().double().cpu(), -1.0)
        if not norm:
            out["dx"] = (g, gm)
        else:
            out["dw"] = ((g * xh).sum((0, 1)), 2 * (gm * xh.abs()).sum((0, 1)))
            h, hm = g * w, gm * w.abs()
            out["dx"] = (rstd * (h - xh * (h * xh).mean(-1, keepdim=True)),
                         2 * rstd * (hm + xh.abs() * (hm * xh.abs()).mean(-1, keepdim=True)))
    return out, 64.0 * U32


# ------------------------------------------------------------------ codes

def e4m3(y):
    """Nearest values of four exponent and three fraction bits, ties to even, at most 448 (float64)."""
    y = np.asarray(y, np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -20))), -6)
    step = 2.0 ** (e - 3)
    return np.clip(np.rint(y / step) * step, -448, 448)


def quantise(x, codes):
    """Values of the codes (float64) and scales (float32) of rows [.., D]; every quotient and product in float32."""
    x = x.detach().float().cpu().numpy()
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1, keepdims=True)
        live = np.isfinite(amax) & (amax >= np.float32(2.0 ** -100))
        top = np.float32(TOP[codes])
        some = np.where(live, amax, np.float32(1))
        y = np.where(live, x, np.float32(0)) * (top / some)
        scale = np.where(live, amax / top, np.where(np.isfinite(amax), np.float32(0), np.float32(np.nan)))
    assert y.dtype == np.float32 and scale.dtype == np.float32
    return np.rint(y).astype(np.float64) if codes == "int8" else e4m3(y), scale[..., 0]


def held(x, codes):
    """Rows as the cache holds them, in float64."""
    if codes is None:
        return x.detach().double().cpu()
    y, scale = quantise(x, codes)
    return torch.from_numpy(y * scale[..., None].astype(np.float64))


def places(table, page_size, row_ptr, lengths):
    """Page and place of each of the call's rows."""
    table = table.cpu().numpy()
    seq = np.repeat(np.arange(len(lengths)), np.diff(row_ptr))
    at = np.concatenate([np.arange(n - c, n) for n, c in zip(lengths, np.diff(row_ptr))] + [np.zeros(0, np.int64)]).astype(np.int64)
    return table[seq, at // page_size], at % page_size


# ------------------------------------------------------------------ attention

def attend(q, k, v, row_ptr, lengths, scale, causal=True, window=0, absent=None):
    """q [n, H, D]; k, v: per sequence [length, Hkv, D] float64; absent: per sequence a bool [length] of missing keys.
    dict name -> (value, magnitudes), and the factor."""
    q = q.detach().double().cpu()
    o, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    G = q.shape[1] // k[0].shape[1]
    smax = 0.0
    for b, n in enumerate(lengths):
        n = int(n)
        r0, r1 = int(row_ptr[b]), int(row_ptr[b + 1])
        for r in range(r0, r1):
            own = n - (r1 - r) if causal else n - 1
            first = max(0, own + 1 - window) if window else 0
            cols = np.arange(first, own + 1)
            if absent is not None:
                cols = cols[~absent[b][cols]]
            if len(cols) == 0:
                continue
            for h in range(q.shape[1]):
                kk, vv = k[b][cols, h // G], v[b][cols, h // G]
                s = kk @ q[r, h] * scale
                if bool(torch.isfinite(s).all()):
                    smax = max(smax, float((kk.abs() @ q[r, h].abs() * abs(scale)).max()))
                p = torch.softmax(s, 0)
                lse[r, h] = torch.logsumexp(s, 0)
                o[r, h], mag[r, h] = p @ vv, p @ vv.abs()
    return {"o": (o, mag), "lse": (lse, torch.full_like(lse, 1 + smax))}, 128.0 * U32 * (1.0 + smax / 8.0)


def check(name, got, ref, factor, rounded=False, more=0.0):
    """|got - value| <= (factor + more) magnitudes (+ a bf16 rounding); infinities and NaN have to match."""
    value, mag = ref
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    odd = ~torch.isfinite(value)
    assert torch.equal(torch.isnan(got[odd]), torch.isnan(value[odd])), name
    assert torch.equal(got[odd & ~torch.isnan(value)], value[odd & ~torch.isnan(value)]), name
    fine = ~odd
    err = (got - value).abs()[fine]
    bound = (factor + more) * mag[fine] + (U16 * value.abs()[fine] if rounded else 0.0) + 1e-37
    bad = ~(err <= bound)
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {worst:.3g} of the tolerance"
    return worst

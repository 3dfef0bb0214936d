"""64-bit references of the context operators, with the magnitudes that bound their rounding errors.

Tolerances.  u = 2^-24 is half a unit of fp32.  A score is an inner product of at most 128 terms plus a bias,
an exponential and a normalisation: 128 u of the sum of the magnitudes covers their roundings while the scores
stay within about 8; larger ones amplify an error of s in exp(s), so the factor grows with max |s| / 8.  Every
output is a sum; its error is taken relative to the same sum over magnitudes (`abs` below), so cancellation
needs no allowance of its own.  bf16 keeps 8 significant bits: half a unit is 2^-8.  bf16 tensors add the rounding
of the output (2^-8 of its value) and of one 16-bit operand of the last product (2^-8 of the magnitudes).
"""
import math

import numpy as np
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8


def bucket(rel, thresholds):
    return np.searchsorted(np.asarray(thresholds, np.int64), np.asarray(rel, np.int64), side="right")


def attention(q, k, v, q_ptr, k_ptr, scale, bias=None, thresholds=None, q_pos=None, k_pos=None, keep=None, d_o=None):
    """dict name -> (value, magnitudes) in float64 on the CPU; with d_o also the gradients."""
    q, k, v = (t.detach().double().cpu() for t in (q, k, v))
    g = None if d_o is None else d_o.detach().double().cpu()
    n_q, H, D = q.shape
    n_k, Hkv, _ = k.shape
    G = H // Hkv
    o, lse = torch.zeros_like(q), torch.full((n_q, H), -math.inf, dtype=torch.float64)
    out = {n: [torch.zeros_like(t), torch.zeros_like(t)] for n, t in (("dq", q), ("dk", k), ("dv", v))}
    oabs = torch.zeros_like(q)
    nb = 0 if bias is None else bias.shape[1]
    db = [torch.zeros((H, nb), dtype=torch.float64) for _ in range(2)]
    smax = 0.0
    for b in range(len(q_ptr) - 1):
        rows = torch.arange(int(q_ptr[b]), int(q_ptr[b + 1]))
        cols = torch.arange(int(k_ptr[b]), int(k_ptr[b + 1]))
        qp = rows - int(q_ptr[b]) if q_pos is None else q_pos.cpu()[rows]
        kp = cols - int(k_ptr[b]) if k_pos is None else k_pos.cpu()[cols]
        if keep is not None:
            kept = keep.cpu()[cols].bool()
            cols, kp = cols[kept], kp[kept]
        if rows.numel() == 0 or cols.numel() == 0:
            continue
        bk = None
        if bias is not None:
            rel = np.clip(kp.numpy().astype(np.int64)[None, :] - qp.numpy().astype(np.int64)[:, None],
                          -2 ** 31, 2 ** 31 - 1)
            bk = torch.from_numpy(bucket(rel, thresholds))
        for h in range(H):
            qh, kh, vh = q[rows, h], k[cols, h // G], v[cols, h // G]
            s = qh @ kh.T * scale
            if bk is not None:
                s = s + bias.double().cpu()[h][bk]
            smax = max(smax, float(s.abs().max()))
            lse[rows, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[rows, h][:, None])
            o[rows, h] = p @ vh
            oabs[rows, h] = p @ vh.abs()
            if g is None:
                continue
            gh = g[rows, h]
            dp = gh @ vh.T
            delta = (gh * o[rows, h]).sum(1, keepdim=True)
            ds = p * (dp - delta)
            da = p * (gh.abs() @ vh.abs().T + (gh.abs() * oabs[rows, h]).sum(1, keepdim=True))
            for name, at, val, mag in (("dq", (rows, h), ds @ kh, da @ kh.abs()),
                                       ("dk", (cols, h // G), ds.T @ qh, da.T @ qh.abs())):
                out[name][0][at] += val * scale
                out[name][1][at] += mag * abs(scale)
            out["dv"][0][cols, h // G] += p.T @ gh
            out["dv"][1][cols, h // G] += p.T @ gh.abs()
            if bk is not None:
                db[0][h] += torch.bincount(bk.reshape(-1), ds.reshape(-1), minlength=nb)
                db[1][h] += torch.bincount(bk.reshape(-1), da.reshape(-1), minlength=nb)
    res = {"o": (o, oabs), "lse": (lse, torch.ones_like(lse) * (1 + smax))}
    if g is not None:
        res.update({n: tuple(t) for n, t in out.items()})
        if bias is not None:
            res["dbias"] = tuple(db)
    return res, 128.0 * U32 * (1.0 + smax / 8.0)


def activation(z, act):
    if act == "ssp":
        return torch.logaddexp(z, torch.zeros_like(z)) - math.log(2.0), torch.sigmoid(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    return z, torch.ones_like(z)


def group_norm(x, ptr, groups, eps, act, gamma=None, beta=None, dy=None):
    """As attention(): outputs y, mean, rstd and with dy the gradients, each with its error scale; the factor
    is 64 u (a value's own roundings and those of sums joined in trees)."""
    x = x.detach().double().cpu()
    n, C = x.shape
    w = C // groups
    gamma = torch.ones(C, dtype=torch.float64) if gamma is None else gamma.double().cpu()
    beta = torch.zeros(C, dtype=torch.float64) if beta is None else beta.double().cpu()
    g = None if dy is None else dy.detach().double().cpu()
    B = len(ptr) - 1
    y, ya, dx, dxa = (torch.zeros_like(x) for _ in range(4))
    mean, rstd = torch.zeros((B, groups), dtype=torch.float64), torch.full((B, groups), eps ** -0.5, dtype=torch.float64)
    dg, dga, db, dba = (torch.zeros(C, dtype=torch.float64) for _ in range(4))
    mean_a = torch.ones_like(mean)
    for b in range(B):
        a, e = int(ptr[b]), int(ptr[b + 1])
        if a == e:
            continue
        part = x[a:e].reshape(e - a, groups, w)
        mu = part.mean((0, 2))
        r = 1 / torch.sqrt(((part - mu[None, :, None]) ** 2).mean((0, 2)) + eps)
        mean[b], rstd[b], mean_a[b] = mu, r, part.abs().mean((0, 2))
        xh = ((part - mu[None, :, None]) * r[None, :, None]).reshape(e - a, C)
        # an error of u |x| in x - mean, scaled by rstd, is what xh carries
        xe = (1 + (part.abs() + part.abs().mean((0, 2))[None, :, None]) * r[None, :, None]).reshape(e - a, C)
        z = xh * gamma + beta
        f, slope = activation(z, act)
        y[a:e], ya[a:e] = f, xe * gamma.abs() + beta.abs() + 1
        if g is None:
            continue
        dz = g[a:e] * slope
        ze = g[a:e].abs() * (1.1 * slope.abs() + ya[a:e])      # act'' is at most 1/2; slopes at most 1.1
        dg += (dz * xh).sum(0)
        dga += (ze * (xh.abs() + xe)).sum(0)
        db += dz.sum(0)
        dba += ze.sum(0)
        h, hh = (dz * gamma).reshape(e - a, groups, w), xh.reshape(e - a, groups, w)
        dx[a:e] = ((h - h.mean((0, 2))[None, :, None] - hh * (h * hh).mean((0, 2))[None, :, None])
                   * r[None, :, None]).reshape(e - a, C)
        ha, xa = (ze * gamma.abs()).reshape(h.shape), (xh.abs() + xe).reshape(h.shape)
        dxa[a:e] = ((ha + ha.mean((0, 2))[None, :, None] + xa * (ha * xa).mean((0, 2))[None, :, None])
                    * r[None, :, None]).reshape(e - a, C)
    # var is a mean of squares; its relative error reaches rstd halved, with that of the differences
    res = {"y": (y, ya), "mean": (mean, mean_a), "rstd": (rstd, rstd * (1 + mean_a * rstd))}
    if g is not None:
        res.update({"dx": (dx, dxa), "dgamma": (dg, dga), "dbeta": (db, dba)})
    return res, 64.0 * U32


def check(name, got, ref, factor, rounded):
    """|got - value| <= factor magnitudes (+ the bf16 roundings); infinities and empty rows have to match."""
    value, mag = ref
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    inf = torch.isinf(value)
    assert torch.equal(got[inf], value[inf]), name
    fine = ~inf
    err = (got - value).abs()[fine]
    bound = factor * mag[fine]
    if rounded:
        bound = bound + U16 * (value.abs() + mag)[fine]
    bad = ~(err <= bound + 1e-37)
    worst = float((err / (bound + 1e-37)).max()) if err.numel() else 0.0
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {worst:.3g} of the tolerance"
    return worst

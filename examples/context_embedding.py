"""Bead embeddings conditioned on a sequence encoder's states, fitted and then run in molecular dynamics.

A bead's first features are its type's row of the embedding table: they do not know the sequence the bead stands
in.  The block below adds what the states of a sequence encoder (one per residue and two special ones, so another
length than the beads) have to say:

    h = Emb[type] + attention(group_norm(Emb[type]) Wq, states Wk, states Wv, bias by chain offset) Wo

It is fitted here to a synthetic target (each bead's row plus a part of its chain neighbours' rows), with the
library's operators forward and backward.  The fitted rows, one per bead, are then the embedding table of an
ordinary model whose bead types are 0 .. N - 1, and velocity Verlet runs on it unchanged.

Usage: python examples/context_embedding.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import schnet_cfconv_force_amd as sn  # noqa: E402
import synth  # noqa: E402


class GroupNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, plan, ws):
        y, saved = sn.group_norm_forward(plan, x, gamma, beta, ws, save=True)
        ctx.save_for_backward(x, gamma, beta, *saved)
        ctx.plan, ctx.ws = plan, ws
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gamma, beta, mean, rstd = ctx.saved_tensors
        dx, dgamma, dbeta = sn.group_norm_backward(ctx.plan, x, gamma, beta, (mean, rstd), dy, ctx.ws)
        return dx, dgamma, dbeta, None, None


class CrossAttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, bias, plan, ws, q_pos, k_pos):
        o, saved = sn.cross_attention_forward(plan, q, k, v, ws, bias=bias, q_pos=q_pos, k_pos=k_pos, save=True)
        ctx.save_for_backward(q, k, v, bias, *saved)
        ctx.plan, ctx.ws, ctx.pos = plan, ws, {"q_pos": q_pos, "k_pos": k_pos}
        return o

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, bias, *saved = ctx.saved_tensors
        grads = sn.cross_attention_backward(ctx.plan, q, k, v, saved, d_o, ctx.ws, bias=bias, **ctx.pos)
        return (*grads, None, None, None, None)


class ContextBlock:
    """The block's plans, workspaces and parameters for one batch of chains."""

    def __init__(self, replica_ptr, state_ptr, n_features: int, n_heads: int = 4, n_groups: int = 8, seed: int = 0):
        self.norm = sn.GroupNorm(replica_ptr, n_features, n_groups, activation="ssp")
        self.norm_ws = sn.group_norm_workspace(self.norm)
        self.attn = sn.CrossAttention(replica_ptr, state_ptr, n_heads, n_heads, n_features // n_heads,
                                      thresholds=sn.relative_thresholds(32, 128))
        self.attn_ws = sn.cross_attention_workspace(self.attn)
        # bead i stands at residue i; state 0 is special, state 1 + i belongs to residue i
        n, m = np.diff(replica_ptr), np.diff(state_ptr)
        self.q_pos = torch.from_numpy(np.concatenate([np.arange(k) for k in n]).astype(np.int32)).cuda()
        self.k_pos = torch.from_numpy(np.concatenate([np.arange(k) - 1 for k in m]).astype(np.int32)).cuda()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        F = n_features
        shape = {"wq": (F, F), "wkv": (F, 2 * F), "wo": (F, F)}
        self.params = {name: torch.randn(s, generator=gen, device="cuda") * F ** -0.5 for name, s in shape.items()}
        self.params["wo"].zero_()                       # the block begins as the identity
        self.params["bias"] = torch.zeros((n_heads, 32), device="cuda")
        self.params["gamma"] = torch.ones(F, device="cuda")
        self.params["beta"] = torch.zeros(F, device="cuda")
        for p in self.params.values():
            p.requires_grad_(True)

    def __call__(self, x, states):
        p, a = self.params, self.attn
        q = GroupNormFn.apply(x, p["gamma"], p["beta"], self.norm, self.norm_ws) @ p["wq"]
        kv = (states @ p["wkv"]).view(a.n_k, 2, a.n_kv_heads, a.head_dim)
        o = CrossAttentionFn.apply(q.view(a.q_shape), kv[:, 0], kv[:, 1], p["bias"], a, self.attn_ws, self.q_pos,
                                   self.k_pos)
        return x + o.reshape(x.shape) @ p["wo"]


def make_inputs(n_replicas: int = 4):
    """Chains of the 269-bead workload, and per chain the states of its sequence (synthetic)."""
    cfg = synth.make_config("batched_replicas", n_replicas=n_replicas)
    F = cfg["hyper"]["n_features"]
    emb = torch.from_numpy(np.asarray(cfg["params"]["emb"], np.float32)).cuda()
    types = torch.from_numpy(cfg["types"].astype(np.int64)).cuda()
    x = emb[types]
    gen = torch.Generator(device="cuda").manual_seed(5)
    mix = torch.randn((F, F), generator=gen, device="cuda") * F ** -0.5
    scale = float(x.std())
    rows, ptr = [], [0]
    for a, b in zip(cfg["replica_ptr"][:-1], cfg["replica_ptr"][1:]):
        special = torch.randn((2, F), generator=gen, device="cuda")
        rows += [special[:1], x[a:b] @ mix / scale, special[1:]]
        ptr.append(ptr[-1] + int(b - a) + 2)
    # the target: a bead's row and a part of its neighbours' along the chain
    target = x.clone()
    for a, b in zip(cfg["replica_ptr"][:-1], cfg["replica_ptr"][1:]):
        target[a + 1:b] += 0.25 * x[a:b - 1]
        target[a:b - 1] += 0.25 * x[a + 1:b]
    return cfg, x, torch.cat(rows), np.asarray(ptr, np.int32), target


def fit(block, x, states, target, steps: int = 200, rate: float = 3e-3):
    """Adam on the mean squared error; returns the losses, relative to the block's first output.

    A bias has to reach about ln(length) to single a neighbour out: it learns at a rate of its own.
    """
    others = [p for name, p in block.params.items() if name != "bias"]
    opt = torch.optim.Adam([{"params": others}, {"params": [block.params["bias"]], "lr": 0.1}], lr=rate)
    losses = []
    for _ in range(steps):
        loss = ((block(x, states) - target) ** 2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    losses = torch.stack(losses)
    return (losses / losses[0]).cpu().numpy()


def model_of_rows(cfg, rows):
    """The model and system whose bead i has the embedding row i."""
    n = len(cfg["types"])
    params = dict(cfg["params"], emb=rows.detach().cpu().numpy())
    hyper = dict(cfg["hyper"], n_types=n)
    return sn.Model(params, hyper), sn.System(cfg["replica_ptr"], np.arange(n), cfg["box"])


def evaluate(model, system, cfg, pos):
    cutoff, capacity = cfg["hyper"]["cutoff"], 200 * len(cfg["types"])
    ws = sn.workspace(model, system, capacity)
    row_ptr, col, rev, n_edges = sn.build_csr_neighbors(system, pos, cutoff, capacity, ws)
    energy, forces = sn.energy_forces(model, system, pos, row_ptr, col, rev, n_edges, ws)
    return energy, forces, ws, capacity


def main():
    cfg, x, states, state_ptr, target = make_inputs()
    block = ContextBlock(cfg["replica_ptr"], state_ptr, cfg["hyper"]["n_features"])
    losses = fit(block, x, states, target)
    print(f"fit: relative error {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    with torch.no_grad():
        rows = block(x, states)
    pos = torch.from_numpy(cfg["pos"]).cuda()
    plain = evaluate(sn.Model(cfg["params"], cfg["hyper"]), sn.System(cfg["replica_ptr"], cfg["types"], cfg["box"]),
                     cfg, pos)
    model, system = model_of_rows(cfg, rows)
    energy, forces, ws, capacity = evaluate(model, system, cfg, pos)
    print("energies by type:    ", [round(v, 4) for v in plain[0].tolist()])
    print("energies conditioned:", [round(v, 4) for v in energy.tolist()])
    vel = torch.from_numpy(np.asarray(cfg["vel"], np.float32)).cuda()
    inv_mass = torch.from_numpy(cfg["inv_mass"]).cuda()
    n_steps = 20
    log = [torch.zeros((n_steps, system.n_replicas), dtype=torch.float64, device="cuda") for _ in range(2)]
    sn.verlet_step(model, system, pos, vel, forces, inv_mass, cfg["dt_fs"], synth.FORCE_TO_ACCEL, n_steps,
                   cfg["hyper"]["cutoff"], capacity, ws, epot_log=log[0], ekin_log=log[1])
    total = (log[0] + log[1]).sum(1)
    print(f"MD: {n_steps} steps, total energy {float(total[0]):.4f} -> {float(total[-1]):.4f}")


if __name__ == "__main__":
    main()

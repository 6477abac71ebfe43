"""Attention of several new tokens per sequence, from its definition in 64 bits.

Each new token attends over the sequence's cached rows and over those of the
sequence's new rows that a 0/1 matrix marks ("10.3 -- KV cache implementation
details", section 5: softmax(q K^T / sqrt(d)) V; section 4.2: query head i
reads KV head i / g).  One sequence and one query head at a time; a row that a
token does not see has no part in its result, whatever the row holds.

Besides the result it returns what an error bound of a finite evaluation needs:
``mass`` = sum_j p_j |V_j| per output element, and ``reach`` = the largest
sum_i |q_i k_i| / sqrt(d) over the rows a token sees.
"""
from __future__ import annotations

import torch


def attend(q, keys, vals, new_keys, new_vals, marks):
    """One sequence: q [H, n, D]; keys, vals [H_kv, c, D]; new_* [H_kv, n, D];
    marks bool [n, n].  Returns (out, mass, reach): [H, n, D] twice, [H, n]."""
    H, n, D = q.shape
    g = H // keys.shape[0]
    c = keys.shape[1]
    see = torch.cat([torch.ones(n, c, dtype=torch.bool, device=q.device), marks.to(q.device)], 1)
    out = torch.zeros(H, n, D, dtype=torch.float64, device=q.device)
    mass, reach = torch.zeros_like(out), torch.zeros(H, n, dtype=torch.float64, device=q.device)
    for h in range(H):
        K = torch.cat([keys[h // g], new_keys[h // g]]).double()
        V = torch.cat([vals[h // g], new_vals[h // g]]).double()
        x = q[h].double()
        s = (x @ K.T / D ** 0.5).masked_fill(~see, -torch.inf)
        p = torch.exp(s - s.amax(1, keepdim=True)).masked_fill(~see, 0.0)
        p = p / p.sum(1, keepdim=True)
        p = torch.where(see.any(1, keepdim=True), p, 0.0)   # a token that sees nothing: zeros
        fine = torch.where(torch.isfinite(V), V, 0.0)
        out[h], mass[h] = p @ fine, p @ fine.abs()
        for j in (~torch.isfinite(V)).any(1).nonzero()[:, 0].tolist():   # reaches the tokens that see it, no others
            out[h][see[:, j]] += torch.where(torch.isfinite(V[j]), 0.0, V[j])
        reach[h] = (x.abs() @ K.abs().T / D ** 0.5).masked_fill(~see, 0.0).amax(1)
    return out, mass, reach


def tolerance(ref, mass, reach, dtype: str, D: int, keys: int):
    """How far an evaluation with fp32 products and sums may be off, element by
    element.

    A score is a sum of D products: off by at most (D + 2) 2^-24 of
    sum |q_i k_i| / sqrt(d) (twice that where the sum truncates), and so, with
    the row maximum's, is the exponent; every probability is then off by twice
    that relative amount, and by the exponential's own 2^-21.  Sums over the
    keys add keys * 2^-24.  A 16-bit cache's probabilities are rounded to its
    type (eps / 2 each), and so is the result."""
    eps = {"bf16": torch.finfo(torch.bfloat16).eps, "fp16": torch.finfo(torch.float16).eps, "fp32": torch.finfo(torch.float32).eps}[dtype]
    rel = 4 * (D + 2) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + 2 * keys * 2.0 ** -24
    if dtype != "fp32":
        rel = rel + eps / 2
    # fp16 results below its normal range round in steps of 2^-24
    return rel * mass + eps / 2 * (ref.abs() + rel * mass) + (2.0 ** -25 if dtype == "fp16" else 0.0)

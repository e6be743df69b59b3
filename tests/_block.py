"""fp64 forms of the norms around the block and of the training step, for the GPU tests, with the
element-wise error each fp32 / bf16 kernel may have.

Every reference returns (value, slack): slack is the sum of the magnitudes of the terms behind each
element times a relative error of the fp32 arithmetic, and a bf16 output may be off by half a step
(2^-8 relative) more.  Gradients come from autograd of the fp64 forward, not from the kernels'
formulas."""
from __future__ import annotations

import torch

import token_permute_grouped_amd as tpg
from tests._gpu import DEV

HALF = 2.0 ** -8   # half a step of bf16, relative
FP32 = 2.0 ** -16  # 256 roundings of fp32: longer than any chain of additions or product here


def bf16(*shape, g, std=1.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(torch.bfloat16)


def routing(T, E, k, g, drop=0.0, zipf=0.0):
    """random topk_w and consistent tables of a routing with dropped slots (CPU)"""
    logits = torch.randn(T, E, generator=g)
    if zipf:
        logits -= zipf * torch.log(1.0 + torch.arange(E))
    w, idx = torch.topk(logits, k)
    w = torch.softmax(w, 1)
    idx = torch.where(torch.rand(T, k, generator=g) < drop, -1, idx)
    return tables(idx, E) + (w,)


def tables(idx, E):
    """offsets [E+1], slot_row [T, k] of expert ids idx [T, k] (-1: dropped), plain Python"""
    S = idx.numel()
    flat = idx.reshape(-1).tolist()
    order = sorted((e, s) for s, e in enumerate(flat) if e >= 0)
    slot_row = torch.full((S,), -1, dtype=torch.int32)
    for r, (_, s) in enumerate(order):
        slot_row[s] = r
    counts = torch.bincount(torch.tensor([e for e in flat if e >= 0], dtype=torch.int64), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    return offsets, slot_row.reshape(idx.shape)


def rms(v, w, eps):
    n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return n if w is None else n * w


def combine(y, slot_row, w):
    """fp64 sum_j w_j y[slot_row] over live slots, and the sum of the terms' magnitudes"""
    out, mag = 0.0, 0.0
    rows = slot_row.long()
    for j in range(rows.shape[1]):
        live = rows[:, j] >= 0
        term = torch.zeros(rows.shape[0], y.shape[1], dtype=torch.float64)
        wj = torch.where(live, w[:, j], 0.0)[:, None]
        term = torch.where(live[:, None], y[rows[:, j].clamp(min=0)], 0.0) * wj
        out, mag = out + term, mag + term.abs()
    return out, mag


def stored_rows(I, il):
    """stored W1 row of every row of [gate | up]"""
    r = torch.arange(2 * I)
    if il == 0:
        return r
    c, up = r % I, r // I
    return c // il * 2 * il + up * il + c % il


def glu(gu, I, il, clamp, kept=None):
    """kept: the bf16 pre-activations whose side of the clamp decides (the clamp's gradient jumps from 1 to 0
    there, so a value that rounding takes across it has another gradient altogether)"""
    a = gu[:, stored_rows(I, il)]
    if clamp > 0 and kept is None:
        a = a.clamp(-clamp, clamp)
    elif clamp > 0:
        kept = kept[:, stored_rows(I, il)]
        a = torch.where(kept.abs() <= clamp, a, clamp * kept.sign())
    g, u = a[:, :I], a[:, I:]
    return g * torch.sigmoid(g) * u


def close(got, ref, slack, what, half=HALF):
    """element-wise: |got - ref| <= half a step of |ref| + slack"""
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values not finite or not written"
    err = (got - ref).abs()
    bound = half * ref.abs() + slack
    bad = err > bound
    worst = (err / bound.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {worst:.3g} times it"
    return worst


def dev(t):
    return None if t is None else t.to(DEV)


def nan(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def workspace(p, which):
    return torch.full((max(1, tpg.moe_call_workspace_bytes(p, which)),), 0xFF, dtype=torch.uint8, device=DEV)

"""The decode operators in 64 bits, written from their definitions, and the
error bounds their tests hold the kernels to (test infrastructure).

Bounds count roundings: a rounding to bf16 is off by at most 2^-8 of the
value, an fp32 sum of n products by at most n 2^-23 of the sum of their
absolute values (2^-23 and not 2^-24 per addition: the tensor core may
truncate where it aligns its terms).
"""
from __future__ import annotations

import math

import torch

U_BF16 = 2.0 ** -8
U_F32 = 2.0 ** -23


def unpack_codes(codes: torch.Tensor) -> torch.Tensor:
    """[E, K/8, N] int32 words -> [E, K, N] codes 0..15."""
    q = codes.cpu().long() & 0xFFFFFFFF
    return torch.stack([(q >> (4 * i)) & 15 for i in range(8)], dim=2).flatten(1, 2)


def pack_codes(c: torch.Tensor) -> torch.Tensor:
    """[E, K, N] codes 0..15 -> [E, K/8, N] int32 words."""
    E, K, N = c.shape
    v = (c.long().view(E, K // 8, 8, N) << (4 * torch.arange(8).view(1, 1, 8, 1))).sum(2)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).int()


def q4_values(codes, scales, group: int) -> torch.Tensor:
    """fp64 [E, K, N] that codes and scales stand for."""
    return (unpack_codes(codes) - 8).double() * scales.cpu().double().repeat_interleave(group, 1)


def quantize(w: torch.Tensor, group: int):
    """(codes 0..15 [E, K, N], scales [E, K/group, N] bf16) of bf16 w, by the definition."""
    E, K, N = w.shape
    v = w.cpu().double().view(E, K // group, group, N)
    s = (v.abs().amax(2) / 7).float().bfloat16()
    f = s.double().unsqueeze(2)
    q = torch.where(f > 0, v / torch.where(f > 0, f, torch.ones_like(f)), torch.zeros_like(v))
    return (q.round().clamp(-8, 7) + 8).long().view(E, K, N), s


def capacity(T, k, E, cf):
    if cf is None or not cf > 0:
        return T * k
    return min(T * k, max(0, math.ceil(cf * T * k / E - 1e-9)))


def gelu(z):
    return z / 2 * torch.special.erfc(-z * math.sqrt(0.5))


def silu(z):
    return z * torch.sigmoid(z)


def route(x, w_router, bias, k, gating):
    """fp64 (logits, ids, weights) of the definition; ties to the lower index."""
    lg = x.cpu().double() @ w_router.cpu().double()
    if bias is not None:
        lg = lg + bias.cpu().double()
    order = torch.sort(lg, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :k], order.values[:, :k]
    return lg, ids, gate(lg, ids, gating)


def gate(lg, ids, gating):
    top = lg.gather(1, ids)
    if gating == 0:
        return torch.softmax(top, 1)
    p = torch.softmax(lg, 1).gather(1, ids)
    return p if gating == 1 else p / p.sum(1, keepdim=True)


def logit_error(x, w_router):
    """Bound of an fp32 logit's error, per (token, expert)."""
    return x.shape[1] * U_F32 * (x.cpu().double().abs() @ w_router.cpu().double().abs()) + 1e-30


def dispatch(ids, E, cap):
    """Serial dispatch: (counts, offsets, perm, slot)."""
    T, k = ids.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if len(rows[e]) < cap:
                rows[e].append(t * k + j)
    slot = torch.full((T * k,), -1, dtype=torch.int32)
    perm = torch.full((T * k,), -1, dtype=torch.int32)
    offsets = [0]
    for r in rows:
        for i in r:
            slot[i] = (perm >= 0).sum()
            perm[slot[i]] = i
        offsets.append(offsets[-1] + len(r))
    return (torch.tensor([len(r) for r in rows], dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32),
            perm, slot.view(T, k))


def experts(x, w1, w2, ids, weights, slot, act):
    """fp64 (y, bound of |y_gpu - y|) given the routing; w1(e), w2(e): fp64
    matrices of expert e."""
    x = x.cpu().double()
    T, H = x.shape
    y = torch.zeros(T, H, dtype=torch.float64)
    err = torch.zeros(T, H, dtype=torch.float64)
    for e in sorted({int(ids[t, j]) for t in range(T) for j in range(ids.shape[1]) if slot[t, j] >= 0}):
        who = [(t, j) for t in range(T) for j in range(ids.shape[1]) if int(ids[t, j]) == e and slot[t, j] >= 0]
        t = torch.tensor([a for a, _ in who])
        w = torch.tensor([float(weights[a, b]) for a, b in who], dtype=torch.float64)[:, None]
        a1, a2 = w1(e), w2(e)
        z, dz = x[t] @ a1, H * U_F32 * (x[t].abs() @ a1.abs())
        if act == "gelu":
            h = gelu(z)
            dh = 1.13 * dz + 4e-7 * z.abs()      # |GELU'| <= 1.13; the erf formula is good to 1.5e-7
        else:
            F = z.shape[1] // 2
            g, u, dg, du = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
            h = silu(g) * u
            dh = 1.1 * dg * (u.abs() + du) + silu(g).abs() * du + 1e-6 * h.abs()  # |SiLU'| <= 1.1
        dh = dh + U_BF16 * (h.abs() + dh)        # h is rounded to bf16
        out = h @ a2
        dout = dh @ a2.abs() + h.shape[1] * U_F32 * ((h.abs() + dh) @ a2.abs())
        y.index_add_(0, t, w * out)
        err.index_add_(0, t, w * dout + (1e-5 + 8 * U_F32) * w * out.abs())  # gate weights good to 1e-5
    return y, err + U_BF16 * (y.abs() + err) + 1e-37

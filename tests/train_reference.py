"""The training operators in 64 bits, written from their definitions, and the
error bounds their tests hold the kernels to (test infrastructure).

Every gradient comes as (value, bound).  Bounds count roundings: a rounding to
bf16 is off by at most 2^-8 of the value, an fp32 sum of n products by at most
n 2^-23 of the sum of their absolute values (2^-23 and not 2^-24 per addition:
the tensor core may truncate where it aligns its terms), and what an operand is
off by goes through a product with the other operand's absolute values.  The
activation functions are held to ACT_ERR of (1 + |z|) per factor: 1.5e-7 of the
erfc formula and a few fp32 units of exp and the quotient, times the factors.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8      # a rounding to bf16
A = 2.0 ** -23     # an fp32 addition
ACT_ERR = 2e-6
TINY = 2.0 ** -120  # below bf16's normal numbers roundings are absolute


def capacity(T, k, E, cf):
    if cf is None or not cf > 0:
        return T * k
    return min(T * k, max(0, math.ceil(cf * T * k / E - 1e-9)))


def dispatch(ids, E, cap):
    """(counts, offsets, perm, slot) of ids [T, k]: expert by expert, tokens
    ascending, the first cap kept."""
    T, k = ids.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if len(rows[e]) < cap:
                rows[e].append(t * k + j)
    flat = [a for r in rows for a in r]
    slot = torch.full((T * k,), -1, dtype=torch.int64)
    for r, a in enumerate(flat):
        slot[a] = r
    counts = torch.tensor([len(r) for r in rows])
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    perm = torch.tensor(flat + [-1] * (T * k - len(flat)), dtype=torch.int64)
    return counts, offsets, perm, slot.view(T, k)


# ------------------------------------------------------- 8-bit activations --

def a8_scales(v):
    """Bytes of bf16 values v [..., C], by the definition: the smallest s with
    max <= 127 * 2^(s - 127), at least 1; 255 for a group with inf or NaN."""
    C = v.shape[-1]
    n = -(-C // 32)
    p = torch.nn.functional.pad(v.double(), (0, 32 * n - C)).unflatten(-1, (n, 32))
    fin = torch.isfinite(p).all(-1)
    m = torch.where(fin, p.abs().amax(-1), torch.zeros(()).double())
    b = torch.ones_like(m, dtype=torch.int64)
    for s in range(1, 255):
        b = torch.where(m > 127 * 2.0 ** (s - 127), torch.full_like(b, s + 1), b)
    return torch.where(fin, b, torch.full_like(b, 255))


def a8_codes(v, b):
    C = v.shape[-1]
    s = torch.exp2((b - 127).double()).repeat_interleave(32, -1)[..., :C]
    lim = torch.where(b == 249, 63.0, 127.0).double().repeat_interleave(32, -1)[..., :C]
    bad = (b == 255).repeat_interleave(32, -1)[..., :C]
    q = (torch.where(bad, torch.zeros(()).double(), v.double()) / s).round()  # half to even
    return torch.minimum(torch.maximum(q, -lim), lim).to(torch.int64)


def a8_values(codes, b):
    C = codes.shape[-1]
    s = torch.exp2(b.double() - 127)
    s = torch.where(b.long() == 255, torch.full_like(s, float("nan")), s)
    return codes.double() * s.repeat_interleave(32, -1)[..., :C]


# ------------------------------------------------------------- activations --

def act(z, gated):
    """h [n, F] and its derivatives by z, as z [n, F] or [n, 2, F]."""
    if not gated:
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a, u = z[:, 0], z[:, 1]
    s = torch.sigmoid(a)
    return a * s * u, torch.stack([u * s * (1 + a * (1 - s)), a * s], 1)


def act_error(z, gated):
    """Bounds of what fp32 evaluation is off by, of h and of the derivatives."""
    if not gated:
        e = ACT_ERR * (1 + z.abs())
        return e, e
    a, u = z[:, 0].abs(), z[:, 1].abs()
    return ACT_ERR * (1 + a) * u, torch.stack([ACT_ERR * (1 + a) ** 2 * u, ACT_ERR * (1 + a)], 1)


def mm(a, ea, b, eb=None):
    """a @ b and its bound for operands off by ea, eb, accumulated in fp32."""
    n = a.shape[-1]
    v = a @ b
    e = (ea if torch.is_tensor(ea) else torch.zeros_like(a)) @ b.abs() + n * A * (a.abs() @ b.abs())
    if eb is not None:
        e = e + a.abs() @ eb
    return v, e


def to_bf16(v, e):
    return v, e * (1 + U) + U * v.abs() + TINY


# ------------------------------------------------------------ the experts' FFN --

def ffn_backward(xp, z, w1, w2, offsets, dY, gated, w=None):
    """Gradients of the experts' FFN on compact rows, from kept z; with w [rows]
    the rows' dY is w times the given one, and dw [rows] is returned too.
    Values fp64, (value, bound) each; row gradients before their rounding."""
    E, F = w2.shape[0], w2.shape[1]
    rows = xp.shape[0]
    dxp = (torch.zeros(xp.shape).double(), torch.zeros(xp.shape).double())
    dw = (torch.zeros(rows).double(), torch.zeros(rows).double())
    dw1 = (torch.zeros(w1.shape).double(), torch.zeros(w1.shape).double())
    dw2 = (torch.zeros(w2.shape).double(), torch.zeros(w2.shape).double())
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        if r.start == r.stop:
            continue
        g, ge = mm(dY[r], 0, w2[e].t())
        h, d = act(z[r], gated)
        he, de = act_error(z[r], gated)
        wr = (torch.ones(r.stop - r.start).double() if w is None else w[r])[:, None]
        hw, hwe = to_bf16(wr * h, wr.abs() * he + 4 * A * (wr * h).abs())
        if gated:
            wd, gd, ged = wr[:, None], g[:, None], ge[:, None]
        else:
            wd, gd, ged = wr, g, ge
        dz = wd * gd * d
        dz, dze = to_bf16(dz, wd.abs() * (ged * d.abs() + gd.abs() * de) + 8 * A * dz.abs())
        dz, dze = dz.flatten(1), dze.flatten(1)
        dw[0][r] = (g * h).sum(1)
        dw[1][r] = (ge * h.abs() + g.abs() * he + F * A * (g * h).abs()).sum(1)
        for out, (v, err) in ((dw2, to_bf16(*mm(hw.t(), hwe.t(), dY[r]))),
                              (dw1, to_bf16(*mm(xp[r].t(), 0, dz, dze)))):
            out[0][e], out[1][e] = v, err
        dxp[0][r], dxp[1][r] = mm(dz, dze, w1[e].t())
    return dict(dxp=dxp, dw1=dw1, dw2=dw2, dw=dw)


# --------------------------------------------------------- router and gate --

def dlogits(ids, w, dw, dwe, gating, probs, E):
    """Gradient of the logits [T, E] and its bound."""
    T, k = ids.shape
    s = (w * dw).sum(1, keepdim=True)
    se = (w.abs() * dwe + (k + 3) * A * (w * dw).abs()).sum(1, keepdim=True)
    z = torch.zeros(T, E).double()
    if gating == 1:
        v = probs * (z.scatter_add(1, ids, dw) - s)
        e = probs * (z.scatter_add(1, ids, dwe + 4 * A * dw.abs()) + se + 4 * A * s.abs()) + 4 * A * v.abs()
    else:
        v = z.scatter_add(1, ids, w * (dw - s))
        e = z.scatter_add(1, ids, w.abs() * (dwe + se + 4 * A * (dw.abs() + s.abs())))
    return v, e


def route_backward(x, wr, dl, dle):
    """dx (before its rounding), dw_router and db from the logits' gradient, which
    the kernels hand on as two bf16 numbers: 2^-16 of it."""
    dle = dle + U * U * dl.abs() + TINY
    dx = mm(dl, dle, wr.t())
    dx = dx[0], dx[1] + dl.shape[1] * A * (dl.abs() @ wr.t().abs())  # twice as many terms
    v, e = mm(x.t(), 0, dl, dle)
    e = e + x.shape[0] * A * (x.t().abs() @ dl.abs())
    T = dl.shape[0]
    return dict(dx=dx, dw_router=to_bf16(v, e), db=(dl.sum(0), (dle + T * A * dl.abs()).sum(0)))


def gate(lg, ids, gating):
    if gating == 0:
        return torch.softmax(torch.gather(lg, 1, ids), 1)
    p = torch.gather(torch.softmax(lg, 1), 1, ids)
    return p if gating == 1 else p / p.sum(1, keepdim=True)


# ----------------------------------------------------------------- the layer --

def layer(x, wr, b, w1, w2, ids, slot, gating, gated):
    """y of the definition for a given choice of experts and of what is kept."""
    T, k = ids.shape
    lg = x @ wr + (0 if b is None else b)
    w = gate(lg, ids, gating)
    y = torch.zeros_like(x)
    for e in range(w2.shape[0]):
        t, j = torch.nonzero((ids == e) & (slot >= 0), as_tuple=True)
        z = x[t] @ w1[e]
        h = act(z.view(len(t), 2, -1) if gated else z, gated)[0]
        y = y.index_add(0, t, w[t, j][:, None] * (h @ w2[e]))
    return y


def layer_backward(x, z, wr, w1, w2, ids, w, probs, offsets, perm, slot, dy, gating, gated):
    """All gradients, with bounds, from kept x and z and the forward's gate weights."""
    T, k = ids.shape
    n = int(offsets[-1])
    a = perm[:n]
    t = a // k
    f = ffn_backward(x[t], z[:n], w1, w2, offsets, dy[t], gated, w.reshape(-1)[a])
    dw = [torch.zeros(T * k).double() for _ in range(2)]
    for i in range(2):
        dw[i][a] = f["dw"][i]
    dl, dle = dlogits(ids, w, dw[0].view(T, k), dw[1].view(T, k), gating, probs, w2.shape[0])
    r = route_backward(x, wr, dl, dle)
    dx, dxe = r["dx"]
    dx, dxe = dx.clone(), dxe.clone()
    dx.index_add_(0, t, f["dxp"][0])
    dxe.index_add_(0, t, f["dxp"][1] + (k + 1) * A * f["dxp"][0].abs())
    return dict(dx=to_bf16(dx, dxe), dw_router=r["dw_router"], dbias=r["db"], dw1=f["dw1"], dw2=f["dw2"])


def inside(got, want, name):
    """Asserts |got - value| <= bound everywhere."""
    v, e = want
    d = (got.detach().cpu().double() - v).abs()
    bad = ~(d <= e)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d / e).nan_to_num(1e30).max()):.3g} "
                           f"of the bound, first at {torch.nonzero(bad)[0].tolist()}")

"""The training operators: what is measured of them, their plain forms and their values in 64 bits.

Five kinds of cases:
  rows       the gradients of the rows' way to the experts and back: of y[t] = sum_j w[t, j] Y[slot[t, j]]
             (dY and dw) and of xp[r] = x[perm[r] / k] (dx);
  pack       activations kept in 8 bits for the backward pass, and read back;
  ffn        the gradients of the experts' FFN on rows grouped by expert, from the kept pre-activations
             z = xp W1 in bf16 or in 8 bits;
  route      the gradients of the router and the gate from those of the gate weights;
  step       a training step of the whole layer: forward, then every gradient (a router bias is one that
             balances the experts and is not trained by gradients).

8-bit activations: groups of 32 along the last dimension (the last one may be shorter) share a power of
two 2^s, s the smallest with max |v| <= 127 * 2^s; a code is v / 2^s rounded half to even (of the largest s
that 16 bits reach, codes stay within 63).  The scale is kept as the byte s + 127, at least 1; a group that
holds an infinity or a NaN has the byte 255 and stands for NaN.
Gated experts keep z as [rows, 2, F], gate first.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the smallest call: the gradients between tokens and expert rows of a tiny layer
        dict(name="rows_tiny", op="rows", T=64, H=128, E=8, k=2, cf=0.0),
        # a long skewed batch with a capacity limit: every fourth assignment dropped
        dict(name="rows_skewed", op="rows", T=8192, H=2048, E=64, k=4, cf=1.2),
        # an odd batch's activations, rows that end inside a group of 32
        dict(name="pack_ragged", op="pack", rows=1111, cols=2744),
        # a prompt's pre-activations of wide experts
        dict(name="pack_wide", op="pack", rows=8192, cols=14336),
        # rows received from another rank for many narrow gated experts, kept in 8 bits
        dict(name="ffn_narrow", op="ffn", rows=2500, H=2048, F=1408, E=64, act="swiglu", bits=8),
        # the FFN of the wide experts on a prompt's rows
        dict(name="ffn_wide", op="ffn", rows=8192, H=4096, F=14336, E=8, act="gelu", bits=16),
        # the router of the sweep's widest choice
        dict(name="route_k8", op="route", T=2048, H=4096, E=128, k=8, gating=0),
        # a softmax over all of an odd number of experts, an odd batch
        dict(name="route_all", op="route", T=333, H=1000, E=13, k=3, gating=1),
        # the smallest layer's training step
        dict(name="step_tiny", op="step", T=64, H=128, F=256, E=8, k=2, act="gelu", gating=0, cf=0.0, bias=False, skew=0.0, bits=16),
        # an odd batch with a capacity limit, sizes that fill no tile, 8 bits kept
        dict(name="step_ragged", op="step", T=333, H=1000, F=2744, E=13, k=3, act="gelu", gating=1, cf=1.2, bias=True, skew=0.0, bits=8),
        # many narrow gated experts, one of them chosen by almost every token
        dict(name="step_skewed", op="step", T=8192, H=2048, F=1408, E=64, k=4, act="swiglu", gating=2, cf=1.2, bias=True, skew=4.0, bits=8),
        # a training step of the wide layer on a prompt's length
        dict(name="step_wide", op="step", T=4096, H=4096, F=14336, E=8, k=2, act="gelu", gating=0, cf=0.0, bias=False, skew=0.0, bits=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = work(listed()[-1])
    while True:
        op = rng.choice(["rows", "pack", "ffn", "ffn", "route", "step", "step", "step"])
        H = 8 * max(1, _log(rng, 64, 4096) // 8)
        F = 8 * max(1, _log(rng, 64, 14336) // 8)
        E = _log(rng, 1, 128)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 8192)
        cf = rng.choice([0.0, 0.0, 1.2, 0.7])
        act = rng.choice(["gelu", "swiglu"])
        bits = rng.choice([8, 16])
        gating = rng.randint(0, 2)
        if op == "rows":
            c = dict(op=op, T=T, H=H, E=E, k=k, cf=cf)
        elif op == "pack":
            c = dict(op=op, rows=T, cols=F)
        elif op == "ffn":
            c = dict(op=op, rows=_log(rng, 1, 16384), H=H, F=F, E=E, act=act, bits=bits)
        elif op == "route":
            c = dict(op=op, T=T, H=H, E=E, k=k, gating=gating)
        else:
            c = dict(op=op, T=T, H=H, F=F, E=E, k=k, act=act, gating=gating, cf=cf, bias=rng.random() < 0.4, skew=rng.choice([0.0, 0.0, 4.0]), bits=bits)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).bfloat16()


def _weights(g, E, K, N):
    w = torch.empty(E, K, N, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e] = torch.randn(K, N, generator=g, device=DEV) / math.sqrt(K)
    return w


def _capacity(T, k, E, cf):
    return min(T * k, math.ceil(cf * T * k / E - 1e-9)) if cf > 0 else T * k


def _dispatch(ids, E, cap):
    """slot [T, k] and counts [E] of a dispatch: the rows of an expert in the order of its tokens."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    first = counts.cumsum(0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(T * k, device=ids.device) - first[flat[order]]
    kept = counts.clamp(max=cap)
    start = kept.cumsum(0) - kept
    slot = torch.where(rank < cap, start[flat] + rank, -1)
    return slot.view(T, k), kept


def _clear_tokens(g, T, H, w_router, bias, k):
    """Tokens whose choice does not hang on the last bits of a logit: those with two of their k + 1 best
    next to each other are drawn again, so that every form chooses the same experts."""
    x = _randn(g, T, H)
    wr = w_router.double()
    for _ in range(30):
        lg = x.double() @ wr
        if bias is not None:
            lg += bias.double()
        top = torch.topk(lg, min(k + 1, lg.shape[1]), dim=1).values
        if top.shape[1] < 2:
            break
        near = (top[:, :-1] - top[:, 1:]).amin(1) < 1e-4
        n = int(near.sum())
        if n == 0:
            break
        x[near] = _randn(g, n, H)
    return x


def _scale_of(v):
    """Exponent bytes of groups v [..., 32] (fp32 or fp64): s + 127."""
    m = v.abs().amax(-1)
    fin = torch.isfinite(v).all(-1)
    f, x = torch.frexp(torch.where(fin, m, 1.0))  # m = f 2^x, f in [0.5, 1)
    s = torch.where(f * 128 <= 127, x - 7, x - 6)
    b = torch.where(m > 0, s + 127, 1).clamp(min=1)
    return torch.where(fin, b, 255)


def _pack(v):
    """(codes, bytes) of v [..., C] in fp32 or fp64."""
    C = v.shape[-1]
    n = -(-C // 32)
    p = torch.nn.functional.pad(v, (0, 32 * n - C)).view(*v.shape[:-1], n, 32)
    b = _scale_of(p)
    lim = torch.where(b == 249, 63.0, 127.0)[..., None]
    q = (p / torch.exp2((b - 127).to(v.dtype))[..., None]).round()
    q = torch.where((b == 255)[..., None], 0.0, torch.minimum(torch.maximum(q, -lim), lim))
    return q.view(*v.shape[:-1], 32 * n)[..., :C].to(torch.int8), b.to(torch.uint8)


def _unpack(codes, b, dtype=torch.float32):
    s = torch.exp2(b.to(dtype) - 127)
    s = torch.where(b == 255, float("nan"), s)
    return codes.to(dtype) * s.repeat_interleave(32, -1)[..., :codes.shape[-1]]


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    st = dict(case=case)
    if op == "rows":
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        score = torch.rand(T, E, generator=g, device=DEV)
        score[:, 0] += 0.7 if c["cf"] else 0.0  # with a capacity, an expert that overflows
        ids = torch.topk(score, k, dim=1).indices
        st["slot"], kept = _dispatch(ids, E, _capacity(T, k, E, c["cf"]))
        st["slot"] = st["slot"].int()
        w = torch.rand(T, k, generator=g, device=DEV) + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
        st["dy"] = _randn(g, T, H)
        st["Y"] = _randn(g, T * k, H)
        st["dxp"] = _randn(g, T * k, H)
        st["dY"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV)  # rows past the kept ones stay
    elif op == "pack":
        # rows of different sizes, some columns far larger than the others, as activations have them
        x = torch.randn(c["rows"], c["cols"], generator=g, device=DEV)
        x *= torch.exp(torch.randn(c["rows"], 1, generator=g, device=DEV))
        x *= torch.where(torch.rand(c["cols"], generator=g, device=DEV) < 0.01, 20.0, 1.0)
        st["x"] = x.bfloat16()
    elif op == "ffn":
        rows, H, F, E = c["rows"], c["H"], c["F"], c["E"]
        gated = c["act"] == "swiglu"
        e = torch.randint(0, E, (rows,), generator=g, device=DEV)
        n = torch.bincount(e, minlength=E)
        st["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
        st["xp"] = _randn(g, rows, H)
        st["w1"] = _weights(g, E, H, 2 * F if gated else F)
        st["w2"] = _weights(g, E, F, H)
        z = torch.randn(rows, *((2, F) if gated else (F,)), generator=g, device=DEV)
        st["z"] = _pack(z) if c["bits"] == 8 else z.bfloat16()
        st["dY"] = _randn(g, rows, H, scale=0.01)
    else:
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        st["w_router"] = _randn(g, H, E, scale=1 / math.sqrt(H))
        if op == "route":
            st["x"] = _randn(g, T, H)
            lg = st["x"].float() @ st["w_router"].float()
            p = torch.softmax(lg, 1)
            top = torch.topk(lg, k, dim=1)
            st["ids"] = top.indices.int()
            st["weights"] = torch.gather(p, 1, top.indices) if c["gating"] == 1 else torch.softmax(top.values, 1)
            st["probs"] = p if c["gating"] == 1 else None
            st["dweights"] = torch.randn(T, k, generator=g, device=DEV)
        else:
            F = c["F"]
            bias = None
            if c["bias"] or c["skew"]:
                bias = 0.3 * torch.randn(E, generator=g, device=DEV)
                bias[0] += c["skew"]
            st["bias"] = bias
            st["w1"] = _weights(g, E, H, 2 * F if c["act"] == "swiglu" else F)
            st["w2"] = _weights(g, E, F, H)
            st["x"] = _clear_tokens(g, T, H, st["w_router"], bias, k)
            st["dy"] = _randn(g, T, H, scale=0.01)
    return st


# -------------------------------------------------------------- plain forms --

def _act(z, gated):
    """h and the factors that take dh to dz, for kept z [n, F] or [n, 2, F]."""
    if not gated:
        phi = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a, u = z[:, 0], z[:, 1]
    s = 1 / (1 + torch.exp(-a))
    return a * s * u, torch.stack([u * s * (1 + a * (1 - s)), a * s], 1)


def _dz(dh, d, gated):
    return (dh[:, None] * d).flatten(1) if gated else dh * d


def _plain_rows(st):
    slot, w, dy = st["slot"].long(), st["weights"], st["dy"].float()
    T, k = slot.shape
    kept = slot >= 0
    rows = torch.where(kept, slot, 0)
    Y, dxp = st["Y"].float(), st["dxp"].float()
    dw = torch.where(kept, (Y[rows] * dy[:, None]).sum(2), 0.0)
    dx = torch.where(kept[..., None], dxp[rows], 0.0).sum(1)
    dY = torch.zeros(T * k + 1, dy.shape[1], device=DEV)
    dY[torch.where(kept, slot, T * k).reshape(-1)] = (dy[:, None] * w[..., None]).reshape(T * k, -1)
    return dict(dY=dY[:-1].bfloat16(), dweights=dw, dx=dx.bfloat16())


def _plain_ffn(st):
    c = st["case"]
    gated = c["act"] == "swiglu"
    o = st["offsets"].tolist()
    dxp = torch.zeros_like(st["xp"])
    dw1, dw2 = torch.zeros_like(st["w1"]), torch.zeros_like(st["w2"])
    for e in range(c["E"]):
        lo, hi = o[e], o[e + 1]
        if lo == hi:
            continue
        z = _unpack(st["z"][0][lo:hi], st["z"][1][lo:hi]) if c["bits"] == 8 else st["z"][lo:hi].float()
        dY = st["dY"][lo:hi].float()
        h, d = _act(z, gated)
        dz = _dz(dY @ st["w2"][e].float().t(), d, gated)
        dw2[e] = h.t() @ dY
        dw1[e] = st["xp"][lo:hi].float().t() @ dz
        dxp[lo:hi] = dz @ st["w1"][e].float().t()
    return dict(dxp=dxp, dw1=dw1, dw2=dw2)


def _dlogits(ids, w, dw, gating, probs):
    s = (w * dw).sum(1, keepdim=True)
    if gating == 1:  # softmax over all experts, the chosen ones' probabilities as they are
        return probs * (torch.zeros_like(probs).scatter(1, ids, dw) - s)
    return torch.zeros(*probs, device=DEV).scatter(1, ids, w * (dw - s))


def _plain_route(st):
    c = st["case"]
    x = st["x"].float()
    dl = _dlogits(st["ids"].long(), st["weights"], st["dweights"], c["gating"], st["probs"] if c["gating"] == 1 else (c["T"], c["E"]))
    return dict(dx=(dl @ st["w_router"].float().t()).bfloat16(), dw_router=(x.t() @ dl).bfloat16(), dbias=dl.sum(0))


def _plain_step(st):
    c = st["case"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    gated = c["act"] == "swiglu"
    x, dy = st["x"].float(), st["dy"].float()
    xk = _unpack(*_pack(x)) if c["bits"] == 8 else x
    # logits in 64 bits, as two of them may be next to each other
    lg = st["x"].double() @ st["w_router"].double()
    if st["bias"] is not None:
        lg = lg + st["bias"].double()
    ids = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
    lg = lg.float()
    top = torch.gather(lg, 1, ids)
    probs = torch.exp(lg - top[:, :1])
    probs = probs / probs.sum(1, keepdim=True)
    if c["gating"] == 1:
        w = torch.gather(probs, 1, ids)
    else:
        w = torch.exp(top - top[:, :1])
        w = w / w.sum(1, keepdim=True)
    slot, kept = _dispatch(ids, E, _capacity(T, k, E, c["cf"]))
    flat = slot.reshape(-1)
    perm = torch.full((T * k + 1,), -1, device=DEV, dtype=torch.int64)
    perm[torch.where(flat >= 0, flat, T * k)] = torch.arange(T * k, device=DEV)
    y = torch.zeros(T, H, device=DEV)
    dx = torch.zeros(T, H, device=DEV)
    dw = torch.zeros(T * k, device=DEV)
    dw1, dw2 = torch.zeros_like(st["w1"]), torch.zeros_like(st["w2"])
    lo = 0
    for e, n in enumerate(kept.tolist()):
        if n == 0:
            continue
        a = perm[lo:lo + n]
        lo += n
        t, we = a // k, w.reshape(-1)[a][:, None]
        w1, w2 = st["w1"][e].float(), st["w2"][e].float()
        z = x[t] @ w1
        if gated:
            z = z.view(n, 2, -1)
        y.index_add_(0, t, we * (_act(z, gated)[0] @ w2))
        z = _unpack(*_pack(z)) if c["bits"] == 8 else z.bfloat16().float()
        h, d = _act(z, gated)
        g = dy[t] @ w2.t()
        dw[a] = (g * h).sum(1)
        dz = _dz(we * g, d, gated)
        dw2[e] = (we * h).t() @ dy[t]
        dw1[e] = xk[t].t() @ dz
        dx.index_add_(0, t, dz @ w1.t())
    dl = _dlogits(ids, w, dw.view(T, k), c["gating"], probs if c["gating"] == 1 else (T, E))
    dx += dl @ st["w_router"].float().t()
    return dict(y=y.bfloat16(), dx=dx.bfloat16(), dw_router=(xk.t() @ dl).bfloat16(), dw1=dw1, dw2=dw2)


def _own(state):
    import mixture_experts_layer_12_gb300 as moe
    c = state["case"]
    op = c["op"]
    if op == "rows":
        dY, dw = moe.combine_backward(state["dy"], state["Y"], state["weights"], state["slot"], dY=state["dY"])
        return dict(dY=dY, dweights=dw, dx=moe.dispatch_rows_backward(state["dxp"], state["slot"]))
    if op == "pack":
        q = moe.quantize_a8(state["x"])
        return dict(values=moe.dequantize_a8(q), scales=q.scales)
    if op == "ffn":
        z = moe.A8Tensor(*state["z"]) if c["bits"] == 8 else state["z"]
        dxp, dw1, dw2 = moe.expert_ffn_backward(state["xp"], z, state["w1"], state["w2"], state["offsets"], state["dY"], act=c["act"])
        return dict(dxp=dxp, dw1=dw1, dw2=dw2)
    if op == "route":
        dx, dw_router, dbias = moe.route_backward(state["x"], state["w_router"], state["ids"], state["weights"], state["dweights"], gating=c["gating"],
                                                  probs=state["probs"])
        return dict(dx=dx, dw_router=dw_router, dbias=dbias)
    layer = state.get("layer")
    if layer is None:  # the layer object that a training program keeps
        layer = state["layer"] = moe.MoETrainLayer(state["w_router"], state["w1"], state["w2"], c["k"], bias=state["bias"], capacity_factor=c["cf"] or None,
                                                   gating=c["gating"], act=c["act"], keep_bits=c["bits"])
    y, saved = layer(state["x"])
    g = layer.backward(saved, state["dy"])
    return dict(y=y, dx=g.dx, dw_router=g.dw_router, dw1=g.dw1, dw2=g.dw2)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rows":
        return _plain_rows(state)
    if op == "pack":
        codes, b = _pack(state["x"].float())
        return dict(values=_unpack(codes, b).bfloat16(), scales=b)
    if op == "ffn":
        return _plain_ffn(state)
    if op == "route":
        return _plain_route(state)
    return _plain_step(state)


# --------------------------------------------------------------------- work --

def work(case):
    c, op = case, case["op"]
    if op == "rows":
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        n = min(T * k, E * _capacity(T, k, E, c["cf"]))  # rows kept, at most
        # dy, the kept rows of Y and dxp in, dY and dx out
        return dict(bytes=2.0 * H * (2 * T + 3 * n) + 12.0 * T * k, flops=4.0 * n * H)
    if op == "pack":  # 16 bits in, 8 out; those in again, 16 bits out
        n = c["rows"] * c["cols"]
        return dict(bytes=n * (6 + 2 / 32), flops=2.0 * n)
    if op == "route":
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        terms = E if c["gating"] == 1 else k
        return dict(bytes=4.0 * T * H + 4.0 * H * E + T * (12.0 * k + (4.0 * E if c["gating"] == 1 else 0)), flops=4.0 * T * H * terms)
    H, F, E = c["H"], c["F"], c["E"]
    n1 = 2 if c["act"] == "swiglu" else 1
    weights = 2.0 * E * H * F * (n1 + 1)
    if op == "ffn":
        n = c["rows"]
        kept = n * F * n1 * (2 if c["bits"] == 16 else 1 + 1 / 32)
        hit = 1 - (1 - 1 / E) ** n
        return dict(bytes=weights * (1 + hit) + kept + 6.0 * n * H, flops=4.0 * n * H * F * (n1 + 1))
    T, k = c["T"], c["k"]
    n = min(T * k, E * _capacity(T, k, E, c["cf"]))
    hit = 1 - (1 - k / E) ** T
    # x, dy, the weights twice (forward and backward) in; y, dx and the gradients out
    return dict(bytes=weights * (1 + 2 * hit) + 8.0 * T * H + 6.0 * H * E, flops=6.0 * n * H * F * (n1 + 1) + 6.0 * T * H * E)


# -------------------------------------------------------------------- exact --

def _kept64(v, bits):
    """What a tensor in 64 bits stands for once it was kept in 16 or 8 bits: group by group."""
    if bits == 16:
        return v.bfloat16().double()  # an even split of 64 bits into 16: rounded once
    parts = []
    for u in v.split(32, -1):
        m = u.abs().amax(-1, keepdim=True)
        step = torch.exp2(torch.ceil(torch.log2(m.clamp(min=1e-300) / 127)).clamp(min=-126.0))
        step = torch.where(m > 127 * step, 2 * step, torch.where((m <= 63.5 * step) & (step > 2.0 ** -126), step / 2, step))
        parts.append((u / step).round() * step)
    return torch.cat(parts, -1)


def _gate64(lg, ids, gating):
    if gating == 0:
        return torch.softmax(torch.gather(lg, 1, ids), 1)
    p = torch.gather(torch.softmax(lg, 1), 1, ids)
    return p if gating == 1 else p / p.sum(1, keepdim=True)


def _h64(z, gated):
    if gated:
        return torch.nn.functional.silu(z[:, 0]) * z[:, 1]
    return z / 2 * torch.special.erfc(-z * math.sqrt(0.5))


def _exact_rows(st):
    slot = st["slot"].cpu().tolist()
    T, k = st["slot"].shape
    dY = torch.zeros(T * k, st["dy"].shape[1], dtype=torch.float64, device=DEV)
    pairs = [(t, j, s) for t in range(T) for j, s in enumerate(slot[t]) if s >= 0]
    t, j, s = (torch.tensor(v, dtype=torch.long, device=DEV) for v in zip(*pairs))
    dy = st["dy"].double()
    dY[s] = dy[t] * st["weights"].double()[t, j][:, None]
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    dw[t, j] = torch.linalg.vecdot(dy[t], st["Y"].double()[s])
    dx = torch.zeros_like(dy)
    for col in range(k):  # one slot of every token at a time
        m = j == col
        dx[t[m]] += st["dxp"].double()[s[m]]
    return dict(dY=dY, dweights=dw, dx=dx)


def _exact_ffn(st):
    c = st["case"]
    gated = c["act"] == "swiglu"
    o = st["offsets"].tolist()
    dxp = torch.zeros(st["xp"].shape, dtype=torch.float64, device=DEV)
    dw1 = torch.zeros(st["w1"].shape, dtype=torch.float64, device=DEV)
    dw2 = torch.zeros(st["w2"].shape, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        if c["bits"] == 8:
            codes, b = st["z"][0][r].double(), st["z"][1][r].double()
            z = torch.cat([codes[..., 32 * i:32 * i + 32] * 2.0 ** (b[..., i:i + 1] - 127) for i in range(b.shape[-1])], -1)
        else:
            z = st["z"][r].double()
        with torch.enable_grad():
            z.requires_grad_()
            w2 = st["w2"][e].double().requires_grad_()
            dz, dw2[e] = torch.autograd.grad(_h64(z, gated) @ w2, (z, w2), st["dY"][r].double())
        dz = dz.flatten(1)
        dw1[e] = st["xp"][r].double().t() @ dz
        dxp[r] = dz @ st["w1"][e].double().t()
    return dict(dxp=dxp, dw1=dw1, dw2=dw2)


def _exact_route(st):
    c = st["case"]
    x, wr = st["x"].double(), st["w_router"].double()
    ids, w = st["ids"].long(), st["weights"].double()
    dw = st["dweights"].double()
    if c["gating"] == 1:  # the Jacobian of a softmax over all experts, column by column of the chosen ones
        p = st["probs"].double()
        dl = torch.zeros_like(p)
        for j in range(c["k"]):
            i = ids[:, j:j + 1]
            dl -= p * w[:, j:j + 1] * dw[:, j:j + 1]
            dl.scatter_add_(1, i, w[:, j:j + 1] * dw[:, j:j + 1])
    else:
        with torch.enable_grad():  # logits that give these weights: their logarithms
            lg = w.log().requires_grad_()
            d, = torch.autograd.grad(torch.softmax(lg, 1), lg, dw)
        dl = torch.zeros(c["T"], c["E"], dtype=torch.float64, device=DEV).scatter(1, ids, d)
    return dict(dx=dl @ wr.t(), dw_router=x.t() @ dl, dbias=dl.sum(0))


def _exact_step(st):
    c = st["case"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    gated = c["act"] == "swiglu"
    x, dy, wr = st["x"].double(), st["dy"].double(), st["w_router"].double()
    xk = _kept64(x, 8) if c["bits"] == 8 else x
    lg = x @ wr
    if st["bias"] is not None:
        lg = lg + st["bias"].double()
    rows = lg.cpu().tolist()
    chosen = [sorted(range(E), key=lambda e: (-v[e], e))[:k] for v in rows]
    ids = torch.tensor(chosen, device=DEV)
    cap = _capacity(T, k, E, c["cf"])
    kept = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if len(kept[chosen[t][j]]) < cap:
                kept[chosen[t][j]].append((t, j))
    w = _gate64(lg, ids, c["gating"])
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    dw1 = torch.zeros(st["w1"].shape, dtype=torch.float64, device=DEV)
    dw2 = torch.zeros(st["w2"].shape, dtype=torch.float64, device=DEV)
    for e in range(E):
        if not kept[e]:
            continue
        t, j = (torch.tensor(v, device=DEV) for v in zip(*kept[e]))
        w1 = st["w1"][e].double()
        z = x[t] @ w1
        if gated:
            z = z.unflatten(1, (2, -1))
        we = w[t, j][:, None]
        w2 = st["w2"][e].double()
        y[t] += we * (_h64(z, gated) @ w2)
        with torch.enable_grad():
            z = _kept64(z, c["bits"]).requires_grad_()
            we, w2 = we.detach().requires_grad_(), w2.requires_grad_()
            dz, dwe, dw2[e] = torch.autograd.grad(we * (_h64(z, gated) @ w2), (z, we, w2), dy[t])
        dw[t, j] = dwe[:, 0]
        dz = dz.flatten(1)
        dw1[e] = xk[t].t() @ dz
        dx[t] += dz @ w1.t()
    with torch.enable_grad():
        leaf = lg.detach().requires_grad_()
        dl, = torch.autograd.grad(_gate64(leaf, ids, c["gating"]), leaf, dw)
    return dict(y=y, dx=dx + dl @ wr.t(), dw_router=xk.t() @ dl, dw1=dw1, dw2=dw2)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        return _exact_rows(st)
    if op == "pack":
        x = st["x"].double()
        return dict(values=_kept64(x, 8), scales=None)
    if op == "ffn":
        return _exact_ffn(st)
    if op == "route":
        return _exact_route(st)
    return _exact_step(st)

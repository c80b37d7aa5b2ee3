"""The decode operators: what is measured of them, their plain forms and their values in 64 bits.

Three kinds of cases:
  layer      a whole MoE layer (router, top-k, gate, dispatch, expert FFN, combine) for a few
             tokens, with bf16 expert weights or with 4-bit ones and group scales;
  matvec     y[r] = x[r] W[e(r)] for a few rows grouped by expert, W in 4 bits with group scales
             (one expert: an ordinary linear layer at decode);
  quantize / dequantize
             bf16 weights to 4 bits with group scales, and back.

4-bit weights of W [E, K, N]: codes [E, K / 8, N] int32, nibble i of a word holds the code of row
8 r + i, code c stands for (c - 8) times the scale of its group; scales [E, K / group, N] bf16.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one user's next token through the layer of the repository's decode workload
        dict(name="layer_t1", op="layer", bits=16, T=1, H=4096, F=14336, E=8, k=2, act="gelu", gating=0, cf=0.0, bias=False, group=0),
        # the smallest call: one token through many narrow gated experts (the skewed workload's widths), a biased router
        dict(name="layer_t1_narrow", op="layer", bits=16, T=1, H=2048, F=1408, E=64, k=4, act="swiglu", gating=2, cf=0.0, bias=True, group=0),
        # an odd batch with a capacity limit, sizes that fill no tile
        dict(name="layer_t13_ragged", op="layer", bits=16, T=13, H=1000, F=2744, E=13, k=3, act="gelu", gating=1, cf=1.2, bias=True, group=0),
        # the same layers with 4-bit experts
        dict(name="layer4_t1", op="layer", bits=4, T=1, H=4096, F=14336, E=8, k=2, act="swiglu", gating=0, cf=0.0, bias=False, group=128),
        dict(name="layer4_t5_narrow", op="layer", bits=4, T=5, H=2048, F=1408, E=64, k=4, act="swiglu", gating=2, cf=0.0, bias=True, group=64),
        dict(name="layer4_t16", op="layer", bits=4, T=16, H=4096, F=14336, E=8, k=2, act="gelu", gating=0, cf=0.0, bias=False, group=128),
        # one linear layer for one token, and expert rows in ragged groups with the finest scales
        dict(name="matvec_1", op="matvec", rows=1, K=4096, N=14336, E=1, group=128, spread=False),
        dict(name="matvec_ragged", op="matvec", rows=37, K=1408, N=2048, E=64, group=32, spread=True),
        # a model's weights quantised once when it is loaded: one narrow layer, one wide one
        dict(name="quantize_narrow", op="quantize", K=1408, N=2048, E=5, group=32),
        dict(name="quantize_wide", op="quantize", K=4096, N=14336, E=4, group=128),
        # 4-bit weights laid out in bf16 for a prompt's large products
        dict(name="dequantize_narrow", op="dequantize", K=2048, N=1408, E=3, group=64),
        dict(name="dequantize_wide", op="dequantize", K=14336, N=4096, E=4, group=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = 1.5e9  # weights of one case, in elements times bytes
    while True:
        op = rng.choice(["layer", "layer", "layer4", "layer4", "matvec", "quantize", "dequantize"])
        group = rng.choice([32, 64, 128])
        E = _log(rng, 1, 128)
        if op in ("layer", "layer4"):
            bits = 4 if op == "layer4" else 16
            step = group if bits == 4 else 8
            H = step * max(1, _log(rng, 64, 8192) // step)
            F = step * max(1, _log(rng, 64, 14336) // step)
            k = rng.randint(1, min(8, E))
            act = rng.choice(["gelu", "swiglu"])
            c = dict(op="layer", bits=bits, T=_log(rng, 1, 64), H=H, F=F, E=E, k=k, act=act, gating=rng.randint(0, 2),
                     cf=rng.choice([0.0, 0.0, 1.2, 0.7]), bias=rng.random() < 0.4, group=group if bits == 4 else 0)
            size = E * H * F * (3 if act == "swiglu" else 2) * 2
        else:
            K = group * max(1, _log(rng, 64, 14336) // group)
            N = 8 * max(1, _log(rng, 64, 14336) // 8)
            if op == "matvec":
                E = E if rng.random() < 0.7 else 1
                c = dict(op=op, rows=_log(rng, 1, 96), K=K, N=N, E=E, group=group, spread=E > 1)
            else:
                c = dict(op=op, K=K, N=N, E=E, group=group)
            size = E * K * N * 2
        if size <= most:
            return c


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _weights(g, E, K, N):
    w = torch.empty(E, K, N, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e] = torch.randn(K, N, generator=g, device=DEV) / math.sqrt(K)
    return w


def _weights4(g, E, K, N, group):
    """Codes and scales as a quantised model has them: normal weights, the largest of a group at code 15 or 1."""
    q = torch.empty(E, K // 8, N, dtype=torch.int32, device=DEV)
    s = torch.empty(E, K // group, N, dtype=torch.bfloat16, device=DEV)
    shift = 4 * torch.arange(8, device=DEV).view(1, 8, 1)
    for e in range(E):
        w = (torch.randn(K, N, generator=g, device=DEV) / math.sqrt(K)).view(K // group, group, N)
        s[e] = (w.abs().amax(1) / 7).bfloat16()
        c = (w / s[e].float()[:, None]).round().clamp(-8, 7).long() + 8
        v = (c.view(K // 8, 8, N) << shift).sum(1)
        q[e] = torch.where(v >= 1 << 31, v - (1 << 32), v).int()
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "layer":
        T, H, F, E, k, group = (case[n] for n in ("T", "H", "F", "E", "k", "group"))
        f1 = 2 * F if case["act"] == "swiglu" else F
        st["x"] = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        st["w_router"] = (torch.randn(H, E, generator=g, device=DEV) / math.sqrt(H)).bfloat16()
        st["bias"] = torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        if case["bits"] == 4:
            st["w1"] = _weights4(g, E, H, f1, group)
            st["w2"] = _weights4(g, E, F, H, group)
        else:
            st["w1"] = _weights(g, E, H, f1)
            st["w2"] = _weights(g, E, F, H)
    elif op == "matvec":
        K, N, E, rows = case["K"], case["N"], case["E"], case["rows"]
        st["x"] = torch.randn(rows, K, generator=g, device=DEV).bfloat16()
        st["w"] = _weights4(g, E, K, N, case["group"])
        if case["spread"]:  # experts of the rows, ascending, as a dispatch leaves them
            e = torch.randint(0, E, (rows,), generator=g, device=DEV)
            n = torch.bincount(e, minlength=E)
        else:
            n = torch.zeros(E, dtype=torch.int64, device=DEV)
            n[0] = rows
        st["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
    elif op == "quantize":
        st["w"] = _weights(g, case["E"], case["K"], case["N"])
    else:
        st["w"] = _weights4(g, case["E"], case["K"], case["N"], case["group"])
    return st


# -------------------------------------------------------------- plain forms --

def _values(q, s, group):
    """[..., K / 8, N] codes and [..., K / group, N] scales -> fp32 [..., K, N]."""
    shift = 4 * torch.arange(8, device=q.device).view(8, 1)
    c = ((q.unsqueeze(-2) >> shift) & 15) - 8
    lead, N = q.shape[:-2], q.shape[-1]
    K = q.shape[-2] * 8
    v = c.reshape(*lead, K // group, group, N).float() * s.float().unsqueeze(-2)
    return v.reshape(*lead, K, N)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    F = z.shape[-1] // 2
    gate, up = z[..., :F], z[..., F:]
    return gate / (1 + torch.exp(-gate)) * up


def _capacity(T, k, E, cf):
    return min(T * k, math.ceil(cf * T * k / E - 1e-9)) if cf > 0 else T * k


def _plain_layer(st):
    c = st["case"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    n = T * k
    x = st["x"].float()
    # logits in 64 bits, as two of them may be next to each other
    logits = (st["x"].double() @ st["w_router"].double()).float()
    if st["bias"] is not None:
        logits = logits + st["bias"]
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :k], order.values[:, :k]
    if c["gating"] == 0:
        ex = torch.exp(top - top[:, :1])
        w = ex / ex.sum(1, keepdim=True)
    else:
        p = torch.exp(top - top[:, :1]) / torch.exp(logits - top[:, :1]).sum(1, keepdim=True)
        w = p if c["gating"] == 1 else p / p.sum(1, keepdim=True)
    # dispatch: rank of every assignment within its expert, the first `cap` kept
    flat = ids.reshape(n)
    cap = _capacity(T, k, E, c["cf"])
    hot = (flat[:, None] == torch.arange(E, device=DEV)).int()
    rank = (hot.cumsum(0) * hot).sum(1) - 1
    counts = hot.sum(0).clamp(max=cap)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    keep = rank < cap
    slot = torch.where(keep, offsets[flat] + rank, -1)
    perm = torch.full((n + 1,), -1, device=DEV, dtype=torch.int64)
    perm = perm.scatter(0, torch.where(keep, slot, n), torch.arange(n, device=DEV))[:n]
    gate = torch.where(keep.view(T, k), w, 0.0)
    # experts: the chosen ones gathered where that is less, else all of them
    if n <= E:
        pick = flat
        rows = x.repeat_interleave(k, 0).unsqueeze(1)
    else:
        pick = slice(None)
        rows = x.unsqueeze(0)
    if c["bits"] == 4:
        w1 = _values(st["w1"][0][pick], st["w1"][1][pick], c["group"])
        z = torch.matmul(rows, w1)
        del w1
        w2 = _values(st["w2"][0][pick], st["w2"][1][pick], c["group"])
    else:
        z = torch.matmul(rows, st["w1"][pick].float())
        w2 = st["w2"][pick].float()
    out = torch.matmul(_act(z, c["act"]), w2)
    if n <= E:
        y = (out.view(T, k, H) * gate[..., None]).sum(1)
    else:
        dense = torch.zeros(T, E, device=DEV).scatter(1, ids, gate)
        y = (out * dense.t()[..., None]).sum(0)
    return dict(y=y.bfloat16(), ids=ids.int(), weights=w, counts=counts.int(), offsets=offsets.int(), perm=perm.int(),
                slot=slot.view(T, k).int())


def _plain_matvec(st):
    c = st["case"]
    x = st["x"].float()
    w = _values(*st["w"], c["group"])
    # all products of rows and experts, then each row's own
    e = torch.searchsorted(st["offsets"][1:].long(), torch.arange(c["rows"], device=DEV), right=True)
    if c["E"] == 1:
        return (x @ w[0]).bfloat16()
    if c["rows"] <= c["E"]:
        return torch.matmul(x.unsqueeze(1), w[e])[:, 0].bfloat16()
    return torch.matmul(x.unsqueeze(0), w)[e, torch.arange(c["rows"], device=DEV)].bfloat16()


def _plain_quantize(st):
    c = st["case"]
    E, K, N, group = c["E"], c["K"], c["N"], c["group"]
    w = st["w"].float().view(E, K // group, group, N)
    s = (w.abs().amax(2) / 7).bfloat16()
    f = s.float().unsqueeze(2)
    q = torch.where(f > 0, (w / f).round().clamp(-8, 7), 0.0)
    return dict(values=(q * f).view(E, K, N).bfloat16(), scales=s)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import mixture_experts_layer_12_gb300 as moe
        if op == "layer":
            layer = state.get("layer")
            if layer is None:  # the layer object that a serving program keeps
                w1, w2 = state["w1"], state["w2"]
                if c["bits"] == 4:
                    w1, w2 = moe.Q4Weights(*w1), moe.Q4Weights(*w2)
                layer = state["layer"] = moe.MoEDecodeLayer(state["w_router"], w1, w2, c["k"], bias=state["bias"], capacity_factor=c["cf"] or None,
                                                            gating=c["gating"], act=c["act"])
            y = layer(state["x"])
            r = layer.routing
            return dict(y=y, ids=r.ids, weights=r.weights, counts=r.counts, offsets=r.offsets, perm=r.perm, slot=r.slot)
        if op == "matvec":
            w = state.get("q4")
            if w is None:
                w = state["q4"] = moe.Q4Weights(*state["w"])
            return moe.matvec_q4(state["x"], w, state["offsets"])
        if op == "quantize":
            q = moe.quantize_q4(state["w"], c["group"])
            return dict(values=moe.dequantize_q4(q), scales=q.scales)
        return moe.dequantize_q4(moe.Q4Weights(*state["w"]))
    if op == "layer":
        return _plain_layer(state)
    if op == "matvec":
        return _plain_matvec(state)
    if op == "quantize":
        return _plain_quantize(state)
    return _values(*state["w"], c["group"]).bfloat16()


# --------------------------------------------------------------------- work --

def work(case):
    c, op = case, case["op"]
    if op == "layer":
        T, H, F, E, k = c["T"], c["H"], c["F"], c["E"], c["k"]
        hit = E * (1 - (1 - k / E) ** T)  # experts with rows, on average
        n1 = 3 if c["act"] == "swiglu" else 2
        per = 2.0 if c["bits"] == 16 else 0.5 + 2.0 / c["group"]
        b = hit * n1 * H * F * per + 2 * H * E + 4 * T * H + 16 * T * k + 8 * E
        return dict(bytes=b, flops=2.0 * T * k * n1 * H * F + 2.0 * T * H * E)
    K, N, E = c["K"], c["N"], c["E"]
    per = 0.5 + 2.0 / c["group"]
    if op == "matvec":
        hit = E * (1 - (1 - 1 / E) ** c["rows"]) if c["spread"] else 1
        return dict(bytes=hit * K * N * per + 2 * c["rows"] * (K + N), flops=2.0 * c["rows"] * K * N)
    if op == "quantize":  # weights in, codes and scales out; those in again, and the values out
        return dict(bytes=E * K * N * (4 + 2 * per), flops=4.0 * E * K * N)
    return dict(bytes=E * K * N * (2 + per), flops=1.0 * E * K * N)


# -------------------------------------------------------------------- exact --

def _exact_w(pair, e, group):
    """fp64 [K, N] of one expert: nibble by nibble."""
    if not isinstance(pair, tuple):
        return pair[e].double()
    q, s = pair[0][e].long() & 0xFFFFFFFF, pair[1][e].double()
    w = torch.empty(q.shape[0] * 8, q.shape[1], dtype=torch.float64, device=DEV)
    for i in range(8):
        w[i::8] = ((q // 16 ** i) % 16 - 8).double()
    return w * s.repeat_interleave(group, 0)


def _exact_layer(st):
    c = st["case"]
    T, H, F, E, k, G = (c[n] for n in ("T", "H", "F", "E", "k", "group"))
    x = st["x"].double()
    lg = (x.cpu() @ st["w_router"].double().cpu())
    if st["bias"] is not None:
        lg = lg + st["bias"].double().cpu()
    rows = lg.tolist()
    ids, w = [], []
    for t in range(T):
        best = sorted(range(E), key=lambda e: (-rows[t][e], e))[:k]
        top = rows[t][best[0]]
        ex = [math.exp(rows[t][e] - top) for e in best]
        z = sum(ex) if c["gating"] == 0 else sum(math.exp(v - top) for v in rows[t])
        p = [v / z for v in ex]
        if c["gating"] == 2:
            p = [v / sum(p) for v in p]
        ids.append(best)
        w.append(p)
    cap = _capacity(T, k, E, c["cf"])
    kept = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if len(kept[ids[t][j]]) < cap:
                kept[ids[t][j]].append((t, j))
    perm, offsets = [], [0]
    slot = [[-1] * k for _ in range(T)]
    y = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        for t, j in kept[e]:
            slot[t][j] = len(perm)
            perm.append(t * k + j)
        offsets.append(len(perm))
        if kept[e]:
            who = torch.tensor([t for t, _ in kept[e]], device=DEV)
            z = x[who] @ _exact_w(st["w1"], e, G)
            if c["act"] == "gelu":
                h = z / 2 * torch.special.erfc(-z * math.sqrt(0.5))
            else:
                h = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:]
            out = h @ _exact_w(st["w2"], e, G)
            scale = torch.tensor([w[t][j] for t, j in kept[e]], dtype=torch.float64, device=DEV)
            y.index_add_(0, who, out * scale[:, None])
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(y=y, ids=as_int(ids), weights=torch.tensor(w, dtype=torch.float64), counts=as_int([len(v) for v in kept]), offsets=as_int(offsets),
                perm=as_int(perm + [-1] * (T * k - len(perm))), slot=as_int(slot))


def exact(case, seed):
    st = prepare(case, seed)
    c, op = case, case["op"]
    if op == "layer":
        return _exact_layer(st)
    if op == "matvec":
        y = torch.empty(c["rows"], c["N"], dtype=torch.float64, device=DEV)
        o = st["offsets"].tolist()
        for e in range(c["E"]):
            if o[e] < o[e + 1]:
                y[o[e]:o[e + 1]] = st["x"][o[e]:o[e + 1]].double() @ _exact_w(st["w"], e, c["group"])
        return y
    if op == "quantize":
        values = torch.empty(c["E"], c["K"], c["N"], dtype=torch.float64, device=DEV)
        scales = torch.empty(c["E"], c["K"] // c["group"], c["N"], dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            w = st["w"][e].double().view(-1, c["group"], c["N"])
            s = (w.abs().amax(1) / 7).bfloat16().double()
            safe = torch.where(s > 0, s, torch.ones_like(s))[:, None]
            values[e] = ((w / safe).round().clamp(-8, 7) * s[:, None]).view(c["K"], c["N"])
            scales[e] = s
        return dict(values=values, scales=scales)
    return torch.stack([_exact_w(st["w"], e, c["group"]) for e in range(c["E"])])

"""The training operators on the GPU against their definition in 64 bits
(tests/train_reference.py, whose bounds count roundings), at the sizes and masks
where they can go wrong, and a run of them together."""
import math
import threading

import pytest
import torch

import mixture_experts_layer_12_gb300 as moe
import train_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_12_gb300 import build
    build.build()
    moe.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF)


def f64(t):
    return t.detach().cpu().double()


def bits_equal(a, b):
    return torch.equal(a.view(torch.uint8 if a.element_size() == 1 else torch.int16 if a.element_size() == 2
                              else torch.int32),
                       b.view(torch.uint8 if b.element_size() == 1 else torch.int16 if b.element_size() == 2
                              else torch.int32))


# ------------------------------------------------------- 8-bit activations --

@pytest.mark.parametrize("shape", [(1, 8), (3, 24), (7, 32), (5, 40), (33, 1000), (2, 3, 72), (129, 2744), (600, 4096),
                                   (1, 31 * 8), (0, 64)])
def test_a8_matches_the_definition(shape):
    g = gen(1)
    x = randn(g, *shape)
    if x.numel():
        x = x * torch.exp(3 * torch.randn(*shape[:-1], 1, generator=g)).to(BF)
    q = moe.quantize_a8(x.to(DEV))
    b = ref.a8_scales(x)
    codes = ref.a8_codes(x, b)
    assert torch.equal(q.scales.cpu().long(), b)
    assert torch.equal(q.codes.cpu().long(), codes)
    assert torch.equal(f64(moe.dequantize_a8(q)), ref.a8_values(codes, b))


def test_a8_special_groups():
    big = torch.finfo(BF).max
    rows = [
        torch.zeros(32), torch.full((32,), -0.0), torch.full((32,), big), torch.full((32,), -big),
        torch.cat([torch.tensor([big, 2.0 ** 126, 1.0]), torch.zeros(29)]),
        torch.cat([torch.tensor([math.inf]), torch.ones(31)]), torch.cat([torch.tensor([-math.inf]), torch.zeros(31)]),
        torch.cat([torch.ones(31), torch.tensor([math.nan])]),
        torch.full((32,), 2.0 ** -133), torch.full((32,), 2.0 ** -126), torch.full((32,), 127 * 2.0 ** -126),
        torch.full((32,), 127.0), torch.full((32,), 127.5), torch.full((32,), 128.0),
        torch.arange(32) * 0.5 + 96.0,  # halves: to even
        torch.cat([torch.tensor([127.0]), torch.arange(31) + 0.5]),
    ]
    x = torch.stack(rows).to(BF)
    q = moe.quantize_a8(x.to(DEV))
    b = ref.a8_scales(x)
    assert torch.equal(q.scales.cpu().long(), b)
    assert torch.equal(q.codes.cpu().long(), ref.a8_codes(x, b))
    got, want = f64(moe.dequantize_a8(q)), ref.a8_values(ref.a8_codes(x, b), b)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.isnan(got[5:8]).all() and torch.isfinite(got[:5]).all()


def test_a8_every_finite_bf16_value():
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    v = v[torch.isfinite(v)]
    v = torch.cat([v, v.new_zeros(-v.numel() % 32)])
    for x in (v.view(-1, 32), v[torch.randperm(v.numel(), generator=gen(2))].view(-1, 32)):
        q = moe.quantize_a8(x.to(DEV))
        b = ref.a8_scales(x)
        assert torch.equal(q.scales.cpu().long(), b)
        assert torch.equal(q.codes.cpu().long(), ref.a8_codes(x, b))
        got = f64(moe.dequantize_a8(q))
        err = (got - x.double()).abs().amax(1)
        s = torch.exp2((b[:, 0] - 127).double())
        assert (err <= torch.where(b[:, 0] == 249, 1.0, 0.5) * s).all()


# ------------------------------------------------------- rows there and back --

def routing(seed, T, E, k, cf=None, skew=0.0):
    g = gen(seed)
    score = torch.rand(T, E, generator=g)
    score[:, 0] += skew
    ids = torch.topk(score, k, dim=1).indices if T else torch.zeros(0, k, dtype=torch.int64)
    counts, offsets, perm, slot = ref.dispatch(ids, E, ref.capacity(T, k, E, cf))
    w = torch.rand(T, k, generator=g) + 0.05
    return ids, w / w.sum(1, keepdim=True), counts, offsets, perm, slot


@pytest.mark.parametrize("T,H,E,k,cf", [(1, 8, 1, 1, None), (1, 128, 8, 8, None), (5, 40, 3, 2, None),
                                        (64, 128, 8, 2, None), (333, 1000, 13, 3, 0.7), (17, 520, 5, 5, 0.4),
                                        (100, 2048, 64, 4, 1.2), (9, 4096, 8, 7, None), (40, 2056, 4, 1, 0.5),
                                        (12, 64, 4, 2, 1e-12)])
def test_combine_and_dispatch_backward(T, H, E, k, cf):
    g = gen(3)
    ids, w, counts, offsets, perm, slot = routing(4, T, E, k, cf, skew=0.5)
    dy, Y, dxp = randn(g, T, H), randn(g, T * k, H), randn(g, T * k, H)
    kept = slot >= 0
    mark = 3.0
    out = torch.full((T * k, H), mark, dtype=BF, device=DEV)
    sl = slot.int().to(DEV)
    dY, dw = moe.combine_backward(dy.to(DEV), Y.to(DEV), w.to(DEV), sl, dY=out)
    assert dY is out
    dx = moe.dispatch_rows_backward(dxp.to(DEV), sl)
    want = torch.full((T * k, H), mark).double()
    bound = torch.zeros(T * k, H).double()
    t, j = torch.nonzero(kept, as_tuple=True)
    want[slot[t, j]] = w.double()[t, j][:, None] * dy.double()[t]
    bound[slot[t, j]] = (ref.U + 2 * ref.A) * want[slot[t, j]].abs() + ref.TINY
    ref.inside(dY, (want, bound), "dY")
    p = dy.double()[:, None] * Y.double()[slot.clamp(min=0)]
    p = torch.where(kept[..., None], p, torch.zeros(()).double())
    ref.inside(dw, (p.sum(2), H * ref.A * p.abs().sum(2)), "dweights")
    s = torch.where(kept[..., None], dxp.double()[slot.clamp(min=0)], torch.zeros(()).double())
    ref.inside(dx, ref.to_bf16(s.sum(1), k * ref.A * s.abs().sum(1)), "dx")
    assert (dw.cpu()[~kept] == 0).all()


def test_rows_of_dropped_slots_do_not_reach_the_gradients():
    T, H, k = 6, 64, 2
    slot = torch.tensor([[0, -1], [-1, -1], [1, 2], [-1, 3], [4, 5], [6, -1]], dtype=torch.int32)
    g = gen(5)
    Y, dxp = randn(g, T * k, H), randn(g, T * k, H)
    Y[7:], dxp[7:] = math.nan, math.nan  # rows that no slot names
    dy = randn(g, T, H)
    dY, dw = moe.combine_backward(dy.to(DEV), Y.to(DEV), torch.full((T, k), 0.5, device=DEV), slot.to(DEV))
    dx = moe.dispatch_rows_backward(dxp.to(DEV), slot.to(DEV))
    assert torch.isfinite(dw).all() and torch.isfinite(dx.float()).all()
    assert (dx[1] == 0).all() and (dw[1] == 0).all()


def test_outputs_over_inputs_are_refused():
    T, H, k = 6, 64, 2
    g = gen(6)
    rows = torch.cat([randn(g, T * k, H), randn(g, T, H)]).to(DEV)  # dxp or Y, dy
    Y, dy = rows[:T * k], rows[T * k:]
    before = rows.clone()
    slot = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    w = torch.full((T, k), 0.5, device=DEV)
    for call in (lambda: moe.dispatch_rows_backward(Y, slot, out=Y[:T]),
                 lambda: moe.dispatch_rows_backward(Y, slot, out=Y[-T:]),
                 lambda: moe.combine_backward(dy, Y, w, slot, dY=Y),
                 lambda: moe.combine_backward(dy, Y, w, slot, dY=rows[T:T + T * k]),
                 lambda: moe.combine_backward(dy, Y, w, slot, dweights=w)):
        with pytest.raises(moe.MoEError, match="overlaps"):
            call()
    q = moe.quantize_a8(Y)
    memory = torch.empty(T * k * H * 2, dtype=torch.uint8, device=DEV)
    q = moe.A8Tensor(memory[:T * k * H].view(torch.int8).view(T * k, H).copy_(q.codes), q.scales)
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.dequantize_a8(q, out=memory.view(BF).view(T * k, H))
    assert torch.equal(rows, before)
    moe.dispatch_rows_backward(Y, slot, out=dy)  # beside one another


# ------------------------------------------------------------- experts' FFN --

def ffn_inputs(seed, counts, H, F, act, bits, lead=0, tail=0):
    """Rows grouped by expert, `lead` before the first and `tail` behind the last."""
    g = gen(seed)
    E = len(counts)
    rows = lead + sum(counts) + tail
    gated = act == "swiglu"
    offsets = lead + torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(counts).cumsum(0)])
    xp, dY = randn(g, rows, H), randn(g, rows, H)
    w1 = randn(g, E, H, 2 * F if gated else F, std=H ** -0.5)
    w2 = randn(g, E, F, H, std=F ** -0.5)
    z = randn(g, *((rows, 2, F) if gated else (rows, F)), std=1.5)
    zk = moe.quantize_a8(z.to(DEV)) if bits == 8 else z.to(DEV)
    zv = f64(moe.dequantize_a8(zk)) if bits == 8 else z.double()
    return offsets, xp, dY, w1, w2, zk, zv


FFN = [
    ([1], 8, 8), ([0], 8, 16), ([3, 0, 2], 64, 64), ([16, 17, 15, 1], 128, 256), ([130, 0, 257, 64], 72, 200),
    ([128, 129, 256, 255], 264, 136), ([300], 520, 392), ([0, 0, 0, 5], 1000, 88), ([2] * 40 + [0] * 3 + [70], 96, 40),
    ([65, 33], 256, 1032), ([600, 7], 128, 128),
    ([2, 0, 1], 72, 4104), ([5], 264, 2056), ([40, 3], 64, 2600),  # K in parts
]


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("counts,H,F", FFN)
def test_expert_ffn_backward(counts, H, F, act, bits):
    offsets, xp, dY, w1, w2, zk, zv = ffn_inputs(11, counts, H, F, act, bits)
    dxp, dw1, dw2 = moe.expert_ffn_backward(xp.to(DEV), zk, w1.to(DEV), w2.to(DEV), offsets.int().to(DEV), dY.to(DEV),
                                            act=act)
    r = ref.ffn_backward(f64(xp), zv, f64(w1), f64(w2), offsets, f64(dY), act == "swiglu")
    ref.inside(dxp, ref.to_bf16(*r["dxp"]), "dxp")
    ref.inside(dw1, r["dw1"], "dw1")
    ref.inside(dw2, r["dw2"], "dw2")
    assert moe.train_status() == 0


@pytest.mark.parametrize("act,bits", [("gelu", 16), ("swiglu", 8), ("gelu", 8), ("swiglu", 16)])
def test_expert_ffn_rows_outside_the_segments(act, bits):
    """Rows before the first segment and behind the last: NaN there reaches
    nothing, and they are left as they are."""
    counts, H, F = [20, 0, 37, 5], 72, 48
    offsets, xp, dY, w1, w2, zk, zv = ffn_inputs(12, counts, H, F, act, bits, lead=3, tail=9)
    n = int(offsets[-1])
    for t in (xp, dY):
        t[:3], t[n:] = math.nan, math.nan
    if bits == 16:
        zk[:3], zk[n:] = math.nan, math.nan
    else:
        zk.scales[:3], zk.scales[n:] = 255, 255
    o = offsets.int().to(DEV)
    dxp, dw1, dw2 = moe.expert_ffn_backward(xp.to(DEV), zk, w1.to(DEV), w2.to(DEV), o, dY.to(DEV), act=act)
    clean = [torch.nan_to_num(f64(t)) for t in (xp, dY)]
    r = ref.ffn_backward(clean[0], torch.nan_to_num(zv), f64(w1), f64(w2), offsets, clean[1], act == "swiglu")
    ref.inside(dxp[3:n], tuple(v[3:n] for v in ref.to_bf16(*r["dxp"])), "dxp")
    ref.inside(dw1, r["dw1"], "dw1")
    ref.inside(dw2, r["dw2"], "dw2")
    Y, z = moe.expert_ffn(xp.to(DEV), w1.to(DEV), w2.to(DEV), o, act=act, keep_bits=bits)
    assert torch.isfinite(Y[3:n].float()).all()
    kept = moe.dequantize_a8(z) if bits == 8 else z
    assert torch.isfinite(kept[3:n].float()).all()


def test_rows_outside_the_segments_with_k_in_parts():
    counts, H, F = [2, 0, 3], 72, 4104
    offsets, xp, dY, w1, w2, zk, zv = ffn_inputs(12, counts, H, F, "gelu", 16, lead=2, tail=4)
    n = int(offsets[-1])
    for t in (xp, dY, zk):
        t[:2], t[n:] = math.nan, math.nan
    dxp, dw1, dw2 = moe.expert_ffn_backward(xp.to(DEV), zk, w1.to(DEV), w2.to(DEV), offsets.int().to(DEV), dY.to(DEV))
    clean = [torch.nan_to_num(f64(t)) for t in (xp, dY)]
    r = ref.ffn_backward(clean[0], torch.nan_to_num(zv), f64(w1), f64(w2), offsets, clean[1], False)
    ref.inside(dxp[2:n], tuple(v[2:n] for v in ref.to_bf16(*r["dxp"])), "dxp")
    ref.inside(dw1, r["dw1"], "dw1")
    ref.inside(dw2, r["dw2"], "dw2")


def test_a_neighbours_nan_and_infinities_stay_its_own():
    counts, H, F = [21, 40, 9], 128, 96
    for bad in (math.nan, math.inf):
        for where in ("xp", "dY", "z"):
            offsets, xp, dY, w1, w2, zk, zv = ffn_inputs(13, counts, H, F, "swiglu", 16)
            lo, hi = int(offsets[1]), int(offsets[2])
            t = dict(xp=xp, dY=dY, z=zk)[where]
            t[lo:hi] = bad
            got = moe.expert_ffn_backward(xp.to(DEV), zk, w1.to(DEV), w2.to(DEV), offsets.int().to(DEV), dY.to(DEV),
                                          act="swiglu")
            xp[lo:hi], dY[lo:hi], zv[lo:hi] = 0, 0, 0
            r = ref.ffn_backward(f64(xp), zv, f64(w1), f64(w2), offsets, f64(dY), True)
            for e in (0, 2):
                s = slice(int(offsets[e]), int(offsets[e + 1]))
                ref.inside(got[0][s], tuple(v[s] for v in ref.to_bf16(*r["dxp"])), "dxp")
                ref.inside(got[1][e], tuple(v[e] for v in r["dw1"]), "dw1")
                ref.inside(got[2][e], tuple(v[e] for v in r["dw2"]), "dw2")
            assert not torch.isfinite((got[1] if where == "xp" else got[2])[1].float()).all()


def test_activations_far_out():
    """Large magnitudes of z: derivatives reach their limits, nothing is 0 times
    infinity."""
    F, H = 64, 32
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 13.0, -13.0, 40.0, -40.0, 88.0, -88.0, 200.0, -200.0,
                      1e4, -1e4]).repeat(4)
    for act in ("gelu", "swiglu"):
        zz = torch.stack([z, torch.ones(F)]) if act == "swiglu" else z
        xp, dY = torch.ones(1, H, dtype=BF), torch.ones(1, H, dtype=BF)
        w1 = torch.ones(1, H, 2 * F if act == "swiglu" else F, dtype=BF)
        w2 = torch.full((1, F, H), 1.0 / H, dtype=BF)
        got = moe.expert_ffn_backward(xp.to(DEV), zz[None].to(BF).to(DEV), w1.to(DEV), w2.to(DEV),
                                      torch.tensor([0, 1], dtype=torch.int32, device=DEV), dY.to(DEV), act=act)
        r = ref.ffn_backward(f64(xp), zz[None].to(BF).double(), f64(w1), f64(w2), torch.tensor([0, 1]), f64(dY),
                             act == "swiglu")
        ref.inside(got[1], r["dw1"], "dw1")
        ref.inside(got[2], r["dw2"], "dw2")
    inf = torch.full((1, 64), math.inf, dtype=BF)  # the limit: GELU'(inf) = 1
    dz = moe.expert_ffn_backward(xp.to(DEV), inf.to(DEV), torch.ones(1, H, 64, dtype=BF, device=DEV), w2.to(DEV),
                                 torch.tensor([0, 1], dtype=torch.int32, device=DEV), dY.to(DEV))[1]
    assert (dz == 1).all()


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("counts,H,F", FFN)
def test_expert_ffn_forward(counts, H, F, act, bits):
    offsets, xp, dY, w1, w2, _, _ = ffn_inputs(14, counts, H, F, act, bits)
    gated = act == "swiglu"
    Y, z = moe.expert_ffn(xp.to(DEV), w1.to(DEV), w2.to(DEV), offsets.int().to(DEV), act=act, keep_bits=bits)
    for e, n in enumerate(counts):
        if n == 0:
            continue
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        zr, ze = ref.mm(f64(xp)[r], 0, f64(w1)[e])
        if gated:
            zr, ze = zr.view(n, 2, F), ze.view(n, 2, F)
        check_kept(z, r, zr, ze, bits)
        check_y(Y[r], zr, ze, f64(w2)[e], gated)


def check_kept(z, r, zr, ze, bits):
    """Kept z against its value zr, known within ze."""
    if bits == 16:
        ref.inside(z[r], ref.to_bf16(zr, ze), "z")
        return
    b = z.scales[r].cpu().long()
    # the scale of some values within the bounds
    lo = ref.a8_scales((zr.abs() - ze).clamp(min=0))
    hi = ref.a8_scales(zr.abs() + ze)
    assert ((b >= lo) & (b <= hi)).all()
    step = torch.exp2((b - 127).double()).repeat_interleave(32, -1)[..., :zr.shape[-1]]
    ref.inside(moe.dequantize_a8(z)[r], (zr, ze + 0.5 * step), "z in 8 bits")


def h_of(zr, ze, gated):
    """The forward's h with its bound, z known within ze; |act'| <= 1.13 (GELU),
    |SiLU'| <= 1.1."""
    h, _ = ref.act(zr, gated)
    he, _ = ref.act_error(zr, gated)
    if gated:
        s = zr[:, 0] * torch.sigmoid(zr[:, 0])
        he = he + 1.1 * ze[:, 0] * (zr[:, 1].abs() + ze[:, 1]) + s.abs() * ze[:, 1]
    else:
        he = he + 1.13 * ze
    return ref.to_bf16(h, he + 4 * ref.A * h.abs())


def check_y(Y, zr, ze, w2, gated):
    h, he = h_of(zr, ze, gated)
    ref.inside(Y, ref.to_bf16(*ref.mm(h, he, w2)), "Y")


# ---------------------------------------------------------- router and gate --

@pytest.mark.parametrize("gating", [0, 1, 2])
@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (1, 64, 8, 2), (3, 40, 5, 5), (64, 128, 8, 2), (333, 1000, 13, 3),
                                     (700, 264, 64, 8), (130, 512, 256, 4), (2049, 128, 100, 1), (17, 2048, 33, 7)])
def test_route_backward(T, H, E, k, gating):
    g = gen(21)
    x, wr = randn(g, T, H), randn(g, H, E, std=H ** -0.5)
    bias = torch.randn(E, generator=g)
    dw = torch.randn(T, k, generator=g)
    lg = f64(x) @ f64(wr) + bias.double()
    ids = torch.topk(lg, k, dim=1).indices
    w = ref.gate(lg, ids, gating).float()
    probs = moe.router_probs(x.to(DEV), wr.to(DEV), bias.to(DEV)) if gating == 1 else None
    if probs is not None:
        want = torch.softmax(lg, 1)
        err = (H * ref.A * (f64(x).abs() @ f64(wr).abs())).amax(1, keepdim=True) + 2e-6
        assert ((f64(probs) - want).abs() <= want * (2 * err + 2e-6) + 1e-30).all()
    dx, dwr, db = moe.route_backward(x.to(DEV), wr.to(DEV), ids.int().to(DEV), w.to(DEV), dw.to(DEV), gating=gating,
                                     probs=probs)
    dl, dle = ref.dlogits(ids, w.double(), dw.double(), torch.zeros(T, k).double(), gating,
                          None if probs is None else f64(probs), E)
    r = ref.route_backward(f64(x), f64(wr), dl, dle)
    ref.inside(dx, ref.to_bf16(*r["dx"]), "dx")
    ref.inside(dwr, r["dw_router"], "dw_router")
    ref.inside(db, r["db"], "dbias")
    if k == 1 and gating != 1:  # a weight of 1 whatever the logits
        assert (dx == 0).all() and (dwr == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T,H,E,k", [(64, 20480, 8, 2), (16, 40000, 24, 3), (5, 30008, 3, 1), (16, 10240, 132, 2)])
def test_route_backward_of_wide_rows(T, H, E, k):
    """More tiles of dW_router than CTA pairs, so that a pair stores several, of
    numbers of columns that do and do not fill their last 32 (E rounded up to 8,
    twice: 16, 48, 16 and 272)."""
    g = gen(24)
    x, wr = randn(g, T, H), randn(g, H, E, std=H ** -0.5)
    dw = torch.randn(T, k, generator=g)
    lg = f64(x) @ f64(wr)
    ids = torch.topk(lg, k, dim=1).indices
    w = ref.gate(lg, ids, 0).float()
    dl, dle = ref.dlogits(ids, w.double(), dw.double(), torch.zeros(T, k).double(), 0, None, E)
    if k == 1:  # weights of 1 have no gradient: of a softmax over all instead
        p = torch.softmax(lg, 1).float()
        dl, dle = ref.dlogits(ids, torch.gather(p, 1, ids).double(), dw.double(), torch.zeros(T, k).double(), 1,
                              p.double(), E)
        w = torch.gather(p, 1, ids)
    r = ref.route_backward(f64(x), f64(wr), dl, dle)
    args = [t.to(DEV) for t in (x, wr, ids.int(), w, dw)]
    first = None
    for _ in range(8):
        got = moe.route_backward(*args, gating=int(k == 1), probs=p.to(DEV) if k == 1 else None)
        ref.inside(got[1], r["dw_router"], "dw_router")
        first = first or got
        assert all(bits_equal(a, b) for a, b in zip(first, got))
    ref.inside(first[0], ref.to_bf16(*r["dx"]), "dx")
    ref.inside(first[2], r["db"], "dbias")
    assert moe.train_status() == 0


# ---------------------------------------------------------------- the layer --

def make_layer(seed, T, H, F, E, k, act="gelu", gating=0, cf=None, bias=False, bits=16, skew=0.0):
    g = gen(seed)
    f1 = 2 * F if act == "swiglu" else F
    x = randn(g, T, H).to(DEV)
    wr = randn(g, H, E, std=H ** -0.5).to(DEV)
    b = torch.randn(E, generator=g) if bias or skew else None
    if skew:
        b[0] += skew
    w1 = randn(g, E, H, f1, std=H ** -0.5).to(DEV)
    w2 = randn(g, E, F, H, std=F ** -0.5).to(DEV)
    dy = randn(g, T, H).to(DEV)
    layer = moe.MoETrainLayer(wr, w1, w2, k, bias=None if b is None else b.to(DEV), capacity_factor=cf, gating=gating,
                              act=act, keep_bits=bits)
    return x, dy, layer


def check_layer(x, dy, layer, y, saved, g):
    """The forward against the definition for its own choice of experts, then the
    gradients against the definition from what was kept."""
    T, k, E = x.shape[0], layer.k, layer.E
    gated = layer.act == "swiglu"
    r = saved.routing
    ids = r.ids.cpu().long()
    counts, offsets, perm, slot = ref.dispatch(ids, E, ref.capacity(T, k, E, layer.capacity_factor))
    for name, want in (("counts", counts), ("offsets", offsets), ("slot", slot)):
        assert torch.equal(getattr(r, name).cpu().long(), want), name
    n = int(offsets[-1])
    assert torch.equal(r.perm.cpu().long()[:n], perm[:n])
    xv, wr, w1, w2 = f64(x), f64(layer.w_router), f64(layer.w1), f64(layer.w2)
    lg = xv @ wr + (0 if layer.bias is None else f64(layer.bias))
    err = (layer.H * ref.A * (xv.abs() @ wr.abs())).amax(1) + 1e-6
    top = torch.sort(lg, 1, descending=True).values
    assert (torch.gather(lg, 1, ids) >= top[:, :k] - 2 * err[:, None]).all()
    w = f64(r.weights)
    ww = ref.gate(lg, ids, layer.gating)
    assert ((w - ww).abs() <= ww * (4 * err[:, None] + 4e-6) + 1e-30).all()
    bits = layer.keep_bits
    if bits == 8:
        b = ref.a8_scales(x.cpu())
        assert torch.equal(saved.x.scales.cpu().long(), b)
        assert torch.equal(saved.x.codes.cpu().long(), ref.a8_codes(x.cpu(), b))
        xk = f64(moe.dequantize_a8(saved.x))
        zk = f64(moe.dequantize_a8(saved.z))
    else:
        assert saved.x is x
        xk, zk = xv, f64(saved.z)
    yv, ye = torch.zeros(T, layer.H).double(), torch.zeros(T, layer.H).double()
    for e in range(E):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        if s.start == s.stop:
            continue
        t, j = perm[s] // k, perm[s] % k
        zr, ze = ref.mm(xv[t], 0, w1[e])
        if gated:
            zr, ze = zr.view(-1, 2, layer.F), ze.view(-1, 2, layer.F)
        check_kept(saved.z, s, zr, ze, bits)
        Y, Ye = ref.mm(*h_of(zr, ze, gated), w2[e])
        we = w[t, j][:, None]
        yv.index_add_(0, t, we * Y)
        ye.index_add_(0, t, we * (Ye + (k + 1) * ref.A * Y.abs()))
    ref.inside(y, ref.to_bf16(yv, ye), "y")
    want = ref.layer_backward(xk, zk, wr, w1, w2, ids, w, None if saved.probs is None else f64(saved.probs), offsets,
                              perm, slot, f64(dy), layer.gating, gated)
    for name in ("dx", "dw_router", "dw1", "dw2") + (("dbias",) if g.dbias is not None else ()):
        ref.inside(getattr(g, name), want[name], name)
    assert moe.moe_get_device_status(layer.status) == 0


LAYERS = [
    dict(T=1, H=8, F=8, E=1, k=1),
    dict(T=1, H=64, F=64, E=8, k=2, act="swiglu"),
    dict(T=2, H=72, F=40, E=3, k=3, gating=1),
    dict(T=64, H=128, F=256, E=8, k=2),
    dict(T=64, H=128, F=256, E=8, k=2, act="swiglu", gating=2, bias=True),
    dict(T=33, H=104, F=88, E=13, k=3, gating=1, cf=1.2, bias=True),
    dict(T=200, H=264, F=136, E=5, k=1, cf=0.6),
    dict(T=150, H=136, F=200, E=64, k=8, act="swiglu", gating=1),
    dict(T=300, H=128, F=64, E=16, k=2, skew=4.0, gating=0),
    dict(T=300, H=128, F=64, E=16, k=4, skew=4.0, cf=0.5, act="swiglu", gating=2),
    dict(T=130, H=72, F=72, E=256, k=8),
    dict(T=40, H=64, F=64, E=4, k=2, cf=1e-12, gating=1),  # everything dropped
    dict(T=700, H=512, F=320, E=4, k=2, act="swiglu"),
    dict(T=3, H=104, F=4136, E=5, k=2, act="swiglu", cf=1.2),  # products with K in parts
    dict(T=2, H=1032, F=1100 // 8 * 8, E=9, k=1, gating=2),
    dict(T=16500, H=64, F=72, E=8, k=2, act="swiglu", gating=1),  # past the one-launch route
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("kw", LAYERS, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_layer_step(kw, bits):
    x, dy, layer = make_layer(31, bits=bits, **kw)
    y, saved = layer(x)
    g = layer.backward(saved, dy, bias_grad=True)
    check_layer(x, dy, layer, y, saved, g)
    assert g.dbias.shape == (layer.E,)
    assert layer.backward(saved, dy).dbias is None


def test_no_tokens():
    for bits in (8, 16):
        for gating in (0, 1):
            x, dy, layer = make_layer(32, T=0, H=64, F=32, E=5, k=2, bits=bits, gating=gating)
            y, saved = layer(x)
            g = layer.backward(saved, dy, bias_grad=True)
            assert y.shape == (0, 64) and g.dx.shape == (0, 64)
            assert (saved.routing.counts == 0).all() and (saved.routing.offsets == 0).all()
            for t in (g.dw_router, g.dw1, g.dw2, g.dbias):
                assert (t == 0).all()
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    w1, w2 = layer.w1, layer.w2
    o = torch.zeros(6, dtype=torch.int32, device=DEV)
    Y, z = moe.expert_ffn(e, w1, w2, o)
    dxp, dw1, dw2 = moe.expert_ffn_backward(e, z, w1, w2, o, e)
    assert (dw1 == 0).all() and (dw2 == 0).all() and Y.shape == dxp.shape == (0, 64)


def test_experts_without_rows_get_zeros():
    x, dy, layer = make_layer(33, T=3, H=64, F=64, E=32, k=2)
    y, saved = layer(x)
    g = layer.backward(saved, dy)
    idle = saved.routing.counts.cpu() == 0
    assert idle.sum() >= 26
    assert (g.dw1[idle.to(DEV)] == 0).all() and (g.dw2[idle.to(DEV)] == 0).all()


def test_forward_agrees_with_the_inference_layer():
    """The same routing, y within the roundings of moe_forward's expert outputs."""
    x, dy, layer = make_layer(34, T=96, H=256, F=320, E=8, k=2)
    y, saved = layer(x)
    other = moe.MoELayer(layer.w_router, layer.w1, layer.w2, 2)
    y2 = other(x)
    assert torch.equal(saved.routing.ids, other.routing.ids)
    assert torch.equal(saved.routing.slot, other.routing.slot)
    assert torch.equal(saved.routing.weights, other.routing.weights)
    assert float((y.float() - y2.float()).norm() / y2.float().norm()) < 2 * ref.U


@pytest.mark.parametrize("gating", [0, 1, 2])
@pytest.mark.parametrize("T,E,k,masked", [(5, 4, 2, (1,)), (200, 13, 3, (0, 5, 12)), (64, 8, 3, (0, 1, 3, 4, 6, 7)),
                                          (150, 130, 6, tuple(range(40, 128)))])
def test_masked_experts(T, E, k, masked, gating):
    """Experts masked by a bias of -inf or NaN, more of them than leave k: chosen
    last, with a weight, a probability and gradients of the logits of 0."""
    x, dy, layer = make_layer(47, T=T, H=128, F=72, E=E, k=k, gating=gating, bias=True)
    runs = []
    for value in (-math.inf, math.nan):
        layer.bias[list(masked)] = value
        y, saved = layer(x)
        g = layer.backward(saved, dy, bias_grad=True)
        if value == -math.inf:
            check_layer(x, dy, layer, y, saved, g)
            off = torch.isin(saved.routing.ids.cpu(), torch.tensor(masked))
            assert (saved.routing.weights.cpu()[off] == 0).all() and off.any() == (E - len(masked) < k)
        probs = moe.router_probs(x, layer.w_router, layer.bias)
        assert (probs[:, list(masked)] == 0).all()
        assert (g.dbias[list(masked)] == 0).all() and (g.dw_router[:, list(masked)] == 0).all()
        runs.append([*all_of(y, saved, g), probs])
    for a, b in zip(*runs):
        assert bits_equal(a, b)


def all_of(y, saved, g):
    z = (saved.z.codes, saved.z.scales) if isinstance(saved.z, moe.A8Tensor) else (saved.z,)
    return [y, g.dx, g.dw_router, g.dbias, g.dw1, g.dw2, *z]


@pytest.mark.parametrize("bits", [16, 8])
def test_same_bits_every_time(bits):
    x, dy, layer = make_layer(35, T=257, H=136, F=264, E=9, k=3, act="swiglu", gating=1, bias=True, bits=bits)
    runs = []
    for _ in range(5):
        y, saved = layer(x)
        runs.append(all_of(y, saved, layer.backward(saved, dy, bias_grad=True)))
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert bits_equal(a.contiguous(), b.contiguous())


def test_several_forwards_before_their_backwards():
    x, dy, layer = make_layer(36, T=70, H=128, F=96, E=6, k=2, bits=8)
    xs = [x, (x * 2).contiguous(), x[:9].contiguous()]
    dys = [dy, dy, dy[:9].contiguous()]
    alone = []
    for a, d in zip(xs, dys):
        y, s = layer(a)
        alone.append(all_of(y, s, layer.backward(s, d, bias_grad=True)))
    fw = [layer(a) for a in xs]
    for i in (2, 0, 1):
        got = all_of(*fw[i], layer.backward(fw[i][1], dys[i], bias_grad=True))
        for a, b in zip(alone[i], got):
            assert bits_equal(a, b)
    again = all_of(*fw[0], layer.backward(fw[0][1], dys[0], bias_grad=True))  # a second time
    for a, b in zip(alone[0], again):
        assert bits_equal(a, b)


def test_changed_inputs_are_refused():
    x, dy, layer = make_layer(37, T=8, H=64, F=64, E=4, k=2)
    y, saved = layer(x)
    x.mul_(2)
    with pytest.raises(ValueError, match="changed"):
        layer.backward(saved, dy)
    y, saved = layer(x)
    layer.w1.mul_(0.5)
    with pytest.raises(ValueError, match="changed"):
        layer.backward(saved, dy)
    layer.keep_bits = 8
    y, saved = layer(x)
    x.mul_(2)  # x was kept in 8 bits: its own memory may be used again
    layer.backward(saved, dy)


def test_streams_and_threads():
    x, dy, layer = make_layer(38, T=120, H=128, F=160, E=8, k=2, act="swiglu", bits=8)
    y, saved = layer(x)
    want = all_of(y, saved, layer.backward(saved, dy, bias_grad=True))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, saved = layer(x, stream=side)
    got = all_of(y, saved, layer.backward(saved, dy, bias_grad=True, stream=side.cuda_stream))
    side.synchronize()
    for a, b in zip(want, got):
        assert bits_equal(a, b)
    fails = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    y, saved = layer(x)
                    got = all_of(y, saved, layer.backward(saved, dy, bias_grad=True))
                    s.synchronize()
                    for a, b in zip(want, got):
                        assert bits_equal(a, b)
        except BaseException as e:  # noqa: BLE001
            fails.append(e)

    ts = [threading.Thread(target=work) for _ in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not fails, fails[0]


def test_captured_steps_replayed_with_other_inputs():
    x, dy, layer = make_layer(39, T=90, H=128, F=96, E=8, k=2, act="swiglu", gating=1, bits=8)
    x2, dy2 = (torch.flip(x, [0]) * 1.5).contiguous(), (torch.flip(dy, [0]) * 0.5).contiguous()
    wants = []
    for a, d in ((x, dy), (x2, dy2)):
        y, s = layer(a)
        wants.append([t.clone() for t in all_of(y, s, layer.backward(s, d, bias_grad=True))])
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn and at once
        xb, db = x.clone(), dy.clone()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, s = layer(xb)
            out = all_of(y, s, layer.backward(s, db, bias_grad=True))
        graphs.append((gr, xb, db, out, (y, s)))
    for order in ((0, 1), (1, 0)):
        for i, (gr, xb, db, out, _) in zip(order, graphs):
            xb.copy_((x, x2)[i])
            db.copy_((dy, dy2)[i])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (gr, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
                gr.replay()
        torch.cuda.synchronize()
        for i, (gr, xb, db, out, _) in zip(order, graphs):
            for a, b in zip(wants[i], out):
                assert bits_equal(a, b)


def test_captured_step_that_holds_x_in_16_bits():
    """x from outside the capture and x made inside it, dropped there and later."""
    x, dy, layer = make_layer(49, T=90, H=128, F=96, E=8, k=2)
    x2 = (x * 1.5).contiguous()
    wants = []
    for a in (x, x2):
        y, s = layer(a)
        wants.append([t.clone() for t in all_of(y, s, layer.backward(s, dy, bias_grad=True))])
    xb = x.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y, s = layer(xb)
        outside = all_of(y, s, layer.backward(s, dy, bias_grad=True))
        inner = xb * 1.5
        y1, s1 = layer(inner)
        del inner
        inside = all_of(y1, s1, layer.backward(s1, dy, bias_grad=True))
    for _ in range(2):
        gr.replay()
        torch.cuda.synchronize()
        for want, got in zip(wants, (outside, inside)):
            for a, b in zip(want, got):
                assert bits_equal(a, b)
    del gr, y, s, y1, s1, outside, inside, xb
    junk = [torch.empty_like(x) for _ in range(4)]
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(layer.status) == 0
    del junk


def test_single_steps_make_the_layers_gradients():
    """dispatch -> expert FFN -> combine and back by the single steps, as a program
    that moves rows between ranks runs them, against the layer's own calls."""
    T, H, F, E, k = 150, 128, 200, 7, 2
    x, dy, layer = make_layer(40, T=T, H=H, F=F, E=E, k=k, act="swiglu", gating=1, cf=0.9, bits=16)
    y, saved = layer(x)
    g = layer.backward(saved, dy, bias_grad=True)
    r, s = saved.routing, saved.shape
    n = T * k
    xp = torch.zeros(n, H, dtype=BF, device=DEV)
    moe.moe_dispatch_rows(s, x, r.perm, r.offsets, xp)
    Y, z = moe.expert_ffn(xp, layer.w1, layer.w2, r.offsets, act="swiglu")
    kept = int(r.offsets[-1])
    assert bits_equal(z[:kept], saved.z[:kept])
    yy = torch.empty(T, H, dtype=BF, device=DEV)
    moe.moe_combine(s, Y, r.weights, r.slot, yy)
    assert float((yy.float() - y.float()).norm() / y.float().norm()) < 2 * ref.U
    dY, dw = moe.combine_backward(dy, Y, r.weights, r.slot)
    dxp, dw1, dw2 = moe.expert_ffn_backward(xp, z, layer.w1, layer.w2, r.offsets, dY, act="swiglu")
    probs = moe.router_probs(x, layer.w_router)
    assert torch.equal(probs, saved.probs)
    dxr, dwr, db = moe.route_backward(x, layer.w_router, r.ids, r.weights, dw, gating=1, probs=probs)
    dx = moe.dispatch_rows_backward(dxp, r.slot).float() + dxr.float()
    # the steps round expert outputs, their gradients and dx's parts to bf16: a few roundings
    for a, b in ((dx, g.dx), (dw1, g.dw1), (dw2, g.dw2), (dwr, g.dw_router), (db, g.dbias)):
        assert float((a.float() - b.float()).norm() / b.float().norm()) < 4 * ref.U


def test_steps_lower_a_loss_like_the_definition_does():
    """A few SGD steps by these calls and by the definition in 64 bits end with
    the same weights, as far as bf16 weights can."""
    T, H, F, E, k = 48, 64, 96, 4, 2
    x, _, layer = make_layer(41, T=T, H=H, F=F, E=E, k=k)
    target = randn(gen(42), T, H).to(DEV)
    master = [f64(t) for t in (layer.w_router, layer.w1, layer.w2)]
    for _ in range(3):
        y, saved = layer(x)
        dy = ((y.float() - target.float()) / (T * H)).to(BF)
        g = layer.backward(saved, dy)
        ids, slot = saved.routing.ids.cpu().long(), saved.routing.slot.cpu().long()
        leaves = [m.clone().requires_grad_() for m in master]
        out = ref.layer(f64(x), leaves[0], None, leaves[1], leaves[2], ids, slot, 0, False)
        gr = torch.autograd.grad(out, leaves, f64(dy))
        for got, want in zip((g.dw_router, g.dw1, g.dw2), gr):
            # from bf16 weights, kept z and bf16 operands: four roundings at most
            assert float((f64(got) - want).norm() / want.norm()) < 4 * ref.U
        for m, t, d in zip(master, (layer.w_router, layer.w1, layer.w2), gr):
            t.copy_((t.double() - 50.0 * d.to(DEV)).to(BF))
            m.copy_(f64(t))


# -------------------------------------------------------- where it can go wrong --

FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
import torch
import mixture_experts_layer_12_gb300 as moe
g = torch.Generator(device="cuda").manual_seed(7)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
x, dy = r(40, 64), r(40, 64)
layer = moe.MoETrainLayer(r(64, 6), r(6, 64, 96), r(6, 48, 64), 2, gating=1, act="swiglu", keep_bits=8)
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    y, saved = layer(x)
    out = layer.backward(saved, dy, bias_grad=True)
gr.replay()
torch.cuda.synchronize()
y2, s2 = layer(x)
want = layer.backward(s2, dy, bias_grad=True)
assert torch.equal(y, y2)
for a, b in zip(out, want):
    assert torch.equal(a, b)
q = moe.quantize_a8(x)
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        moe.MoETrainLayer(layer.w_router, layer.w1, layer.w2, 2, act="swiglu")
except RuntimeError as e:
    assert "outside a capture" in str(e), e
else:
    raise AssertionError("not refused")
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        moe.router_probs(x, layer.w_router)
except RuntimeError as e:
    assert "train_status" in str(e), e
else:
    raise AssertionError("not refused")
torch.cuda.synchronize()
assert moe.train_status() == 0
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    p = moe.router_probs(x, layer.w_router)
gr.replay()
torch.cuda.synchronize()
assert torch.equal(p, moe.router_probs(x, layer.w_router))
print("ok")
"""


def test_a_process_whose_first_calls_are_captured():
    """Nothing of the library has run before the capture: kernels are loaded and
    set up inside it.  A function without a layer needs its status block first."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_backward_on_another_stream_than_the_forward():
    """What a forward kept is not given out again while another stream's backward
    reads it."""
    x, dy, layer = make_layer(43, T=500, H=512, F=512, E=8, k=2, act="swiglu", bits=8)
    y, saved = layer(x)
    want = all_of(y, saved, layer.backward(saved, dy, bias_grad=True))
    want = [t.clone() for t in want]
    side = torch.cuda.Stream()
    for _ in range(10):
        y, saved = layer(x)
        z = [saved.z.codes.numel(), saved.z.scales.numel()]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            g = layer.backward(saved, dy, bias_grad=True)
        del saved  # its memory goes back to the first stream's pool
        junk = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in z for _ in range(2)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(want[1:6], (g.dx, g.dw_router, g.dbias, g.dw1, g.dw2)):
            assert bits_equal(a, b)
        del junk


@pytest.mark.parametrize("forward_beside", [False, True])
def test_x_that_only_the_forward_still_holds(forward_beside):
    """x kept as it is (16 bits) and dropped by its maker is what the forward kept
    as well: not given out again while a backward on another stream than x's reads it."""
    x, dy, layer = make_layer(48, T=500, H=512, F=128, E=8, k=2)
    y, saved = layer(x)
    want = [t.clone() for t in layer.backward(saved, dy, bias_grad=True)]
    side = torch.cuda.Stream()
    for _ in range(10):
        other = x.clone()
        if not forward_beside:
            y, saved = layer(other)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            if forward_beside:
                y, saved = layer(other)
            torch.cuda._sleep(2_000_000)
            g = layer.backward(saved, dy, bias_grad=True)
        del saved, other
        junk = [torch.full_like(x, 77.0) for _ in range(2)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(want, g):
            assert bits_equal(a, b)
        del junk


def test_offsets_that_are_no_dispatch_are_an_error():
    """Offsets that run backwards, overlap or pass the rows are cut on the device
    and reported."""
    rows, H, F, E = 64, 64, 96, 6
    g = gen(44)
    xp, dY = randn(g, rows, H).to(DEV), randn(g, rows, H).to(DEV)
    w1, w2 = randn(g, E, H, F, std=0.1).to(DEV), randn(g, E, F, H, std=0.1).to(DEV)
    z = randn(g, rows, F).to(DEV)
    for o in ([0, 70, 80, 90, 100, 110, 120], [0, 64, 0, 64, 0, 64, 0], [-5, 3, 3, 2, 9, 1, 64], [5, 4, 3, 2, 1, 0, -1]):
        o = torch.tensor(o, dtype=torch.int32, device=DEV)
        for call in (lambda: moe.expert_ffn_backward(xp, z, w1, w2, o, dY),
                     lambda: moe.expert_ffn(xp, w1, w2, o, keep_bits=8)):
            out = call()
            with pytest.raises(moe.MoEError):
                moe.train_status()
        dxp, dw1, dw2 = moe.expert_ffn_backward(xp, z, w1, w2, o, dY)
        assert torch.isfinite(dw1.float()).all() and torch.isfinite(dw2.float()).all()
        with pytest.raises(moe.MoEError):
            moe.train_status()
    assert moe.train_status() == 0


def test_eager_forward_and_captured_backward():
    x, dy, layer = make_layer(45, T=100, H=128, F=96, E=8, k=2, bits=8, gating=1)
    y, saved = layer(x)
    want = layer.backward(saved, dy, bias_grad=True)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        g = layer.backward(saved, dy, bias_grad=True)
    gr.replay()
    gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, g):
        assert bits_equal(a, b)
    saved.shape.T = 3  # a copy: the next call of this size is not touched
    y2, _ = layer(x)
    assert bits_equal(y, y2)


class Layer(torch.autograd.Function):
    """What a program that uses torch's autograd puts around the calls."""

    @staticmethod
    def forward(ctx, x, w_router, w1, w2, layer):
        y, ctx.saved = layer(x.detach())
        ctx.layer = layer
        return y

    @staticmethod
    def backward(ctx, dy):
        g = ctx.layer.backward(ctx.saved, dy.contiguous())
        return g.dx, g.dw_router, g.dw1, g.dw2, None


def test_calls_inside_an_autograd_function():
    x, dy, layer = make_layer(46, T=64, H=128, F=96, E=8, k=2, act="swiglu")
    y, saved = layer(x)
    want = layer.backward(saved, dy)
    leaves = [t.clone().requires_grad_() for t in (x, layer.w_router, layer.w1, layer.w2)]
    layer2 = moe.MoETrainLayer(*[t.detach() for t in leaves[1:]], 2, act="swiglu")
    out = Layer.apply(*leaves, layer2)
    assert bits_equal(out.detach(), y)
    out.backward(dy)
    for t, g in zip(leaves, (want.dx, want.dw_router, want.dw1, want.dw2)):
        assert bits_equal(t.grad, g)


def test_wide_rows_of_codes_past_two_to_the_31():
    """Element offsets past 32 bits."""
    rows, cols = 70000, 32768
    x = torch.zeros(rows, cols, dtype=BF, device=DEV)
    x[-1] = torch.arange(cols, device=DEV).to(BF)
    x[66000, :64] = 3.0
    q = moe.quantize_a8(x)
    assert int(q.codes[66000, :64].float().sum()) == 64 * 96 and int(q.codes[65999].abs().max()) == 0
    b = ref.a8_scales(x[-1:].cpu())
    assert torch.equal(q.scales[-1:].cpu().long(), b)
    assert torch.equal(q.codes[-1:].cpu().long(), ref.a8_codes(x[-1:].cpu(), b))
    v = moe.dequantize_a8(q)
    assert torch.equal(f64(v[-1:]), ref.a8_values(ref.a8_codes(x[-1:].cpu(), b), b))
    assert float(v[66000, 0]) == 3.0 and float(v[:66000].abs().max()) == 0.0


def test_the_longest_rows_of_codes():
    """The largest number of columns that is a multiple of 8 and none of 32."""
    cols = 2 ** 31 - 8
    x = torch.zeros(cols, dtype=BF, device=DEV)
    x[-24:] = torch.arange(24, device=DEV).to(BF)
    x[:8] = 127.0
    q = moe.quantize_a8(x)
    assert q.scales.numel() == 2 ** 26
    assert q.scales[-1] == 125 and q.scales[0] == 127  # 23 > 127 / 8
    assert torch.equal(q.codes[-24:].float() * 2.0 ** (int(q.scales[-1]) - 127), x[-24:].float())
    v = moe.dequantize_a8(q)
    assert bits_equal(v[-24:], x[-24:]) and bits_equal(v[:32], x[:32])
    assert int(torch.count_nonzero(v)) == 23 + 8


@pytest.mark.parametrize("bits", [16, 8])
def test_rows_whose_z_lies_past_two_to_the_31(bits):
    """The last rows of a long batch, whose kept z is past 2^31 elements, come out
    as they do alone."""
    rows, H, F, n = 80000, 64, 14336, 200
    g = gen(50)
    w1 = randn(g, 1, H, 2 * F, std=H ** -0.5).to(DEV)
    w2 = randn(g, 1, F, H, std=F ** -0.5).to(DEV)
    tail_x, tail_d = randn(g, n, H).to(DEV), randn(g, n, H).to(DEV)
    xp, dY = (torch.zeros(rows, H, dtype=BF, device=DEV) for _ in range(2))
    xp[-n:], dY[-n:] = tail_x, tail_d
    out = []
    for x, d in ((xp, dY), (tail_x, tail_d)):
        o = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=DEV)
        Y, z = moe.expert_ffn(x, w1, w2, o, act="swiglu", keep_bits=bits)
        grads = moe.expert_ffn_backward(x, z, w1, w2, o, d, act="swiglu")
        kept = z.codes if bits == 8 else z
        assert kept.numel() > 1 << 31 or x is tail_x
        out.append((Y[-n:].clone(), kept[-n:].clone(), grads[0][-n:].float(), grads[1].float(), grads[2].float()))
    (Y, z, dx, dw1, dw2), (Y1, z1, dx1, e1, e2) = out
    assert bits_equal(Y, Y1) and bits_equal(z, z1)
    # dxp in another number of parts, the weights' over rows of zeros besides
    for a, b in ((dx, dx1), (dw1, e1), (dw2, e2)):
        assert float((a - b).norm() / b.norm()) < ref.U

"""The decode operators on the GPU against their definition in 64 bits
(tests/decode_reference.py, whose bounds count roundings), at the sizes where
they can go wrong, and a run of them together."""
import copy
import math
import threading

import pytest
import torch

import decode_reference as ref
import mixture_experts_layer_12_gb300 as moe

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


def random_q4(g, E, K, N, group):
    """Any codes (0 and 15 too), scales of both signs and zero among them."""
    codes = torch.randint(0, 16, (E, K, N), generator=g)
    s = torch.randn(E, K // group, N, generator=g) / (4 * math.sqrt(K))
    s[torch.rand(s.shape, generator=g) < 0.02] = 0.0
    return moe.Q4Weights(ref.pack_codes(codes).to(DEV), s.to(BF).to(DEV))


def matrices(w, group):
    """e -> fp64 matrix of expert e, of a bf16 tensor or a Q4Weights."""
    if isinstance(w, moe.Q4Weights):
        return lambda e: ref.q4_values(w.codes[e:e + 1], w.scales[e:e + 1], group)[0]
    return lambda e: w[e].cpu().double()


def make_layer(seed, T, H, F, E, k, act="gelu", gating=0, cf=None, bias=False, group=0):
    g = gen(seed)
    f1 = 2 * F if act == "swiglu" else F
    x = randn(g, T, H).to(DEV)
    wr = randn(g, H, E, std=H ** -0.5).to(DEV)
    b = torch.randn(E, generator=g).to(DEV) if bias else None
    if group:
        w1, w2 = random_q4(g, E, H, f1, group), random_q4(g, E, F, H, group)
    else:
        w1 = randn(g, E, H, f1, std=H ** -0.5).to(DEV)
        w2 = randn(g, E, F, H, std=F ** -0.5).to(DEV)
    layer = moe.MoEDecodeLayer(wr, w1, w2, k, bias=b, capacity_factor=cf, gating=gating, act=act)
    return x, layer


def check_routing(x, layer, r):
    """ids exact unless two logits are closer than their error bound; then
    counts, offsets, perm and slot exact for the GPU's ids.  Returns the gate
    weights of the definition at those ids."""
    T, E, k = x.shape[0], layer.E, layer.k
    lg, ids, _ = ref.route(x, layer.w_router, layer.bias, k, layer.gating)
    err = ref.logit_error(x, layer.w_router).amax(1)
    got = r.ids.cpu().long()
    vals = torch.sort(lg, 1, descending=True).values
    near = (vals[:, :min(k, E - 1)] - vals[:, 1:min(k, E - 1) + 1]).amin(1) <= 2 * err if E > 1 else torch.zeros(T, dtype=bool)
    assert torch.equal(got[~near], ids[~near])
    for t in torch.nonzero(near).flatten().tolist():  # a valid choice within the error
        assert len(set(got[t].tolist())) == k and ((got[t] >= 0) & (got[t] < E)).all()
        assert (lg[t, got[t]] >= vals[t, :k] - 2 * err[t]).all()
    want = ref.gate(lg, got, layer.gating)
    # relative error of a weight: exp of logits that are each off by err
    rel = torch.expm1(4 * err)[:, None] + 1e-6
    assert ((r.weights.cpu().double() - want).abs() <= rel * want + 1e-30).all()
    cap = ref.capacity(T, k, E, layer.capacity_factor)
    counts, offsets, perm, slot = ref.dispatch(got, E, cap)
    assert torch.equal(r.counts.cpu(), counts) and torch.equal(r.offsets.cpu(), offsets)
    assert torch.equal(r.perm.cpu()[:T * k], perm) and torch.equal(r.slot.cpu(), slot)
    return got, want, slot


def check_layer(x, layer, y=None):
    y = layer(x) if y is None else y
    r = layer.routing
    assert moe.moe_get_device_status(layer.ws) == 0
    ids, w, slot = check_routing(x, layer, r)
    group = layer.w1.group if layer.q4 else 0
    want, err = ref.experts(x, matrices(layer.w1, group), matrices(layer.w2, group), ids, w, slot, layer.act)
    d = (y.cpu().double() - want).abs()
    assert (d <= err).all(), f"{float((d / err).max())} times the bound"
    return y


# ------------------------------------------------------------------ layers --

LAYERS = [
    # T, H, F, E, k, act, gating, cf, bias
    (1, 64, 64, 1, 1, "gelu", 0, None, False),
    (1, 8, 8, 2, 1, "gelu", 0, None, False),            # below every tile
    (1, 4096, 256, 8, 2, "gelu", 0, None, False),       # one item split over many CTAs
    (1, 256, 4096, 8, 2, "swiglu", 0, None, True),
    (3, 1000, 72, 13, 3, "swiglu", 1, None, True),      # E % 8 != 0, ragged everything
    (5, 520, 1416, 64, 4, "gelu", 2, None, True),
    (7, 128, 256, 256, 8, "gelu", 0, None, False),
    (8, 136, 264, 5, 5, "swiglu", 1, None, False),      # k = E
    (9, 128, 256, 8, 2, "gelu", 0, 0.5, False),         # drops
    (16, 2048, 200, 24, 3, "gelu", 0, None, False),
    (17, 72, 1000, 7, 2, "swiglu", 2, 1.0, True),
    (33, 320, 96, 100, 6, "gelu", 0, None, False),
    (64, 128, 256, 8, 2, "gelu", 0, None, False),       # the tiny workload
    (64, 96, 320, 256, 8, "swiglu", 0, 0.7, True),
    (64, 264, 136, 1, 1, "gelu", 0, None, False),       # 64 rows in one expert
]


@pytest.mark.parametrize("T,H,F,E,k,act,gating,cf,bias", LAYERS)
def test_layer_against_the_definition(T, H, F, E, k, act, gating, cf, bias):
    check_layer(*make_layer(T + H + E, T, H, F, E, k, act, gating, cf, bias))


@pytest.mark.parametrize("T,H,F,E,k,gating,cf,bias", [
    (1, 2048, 2816, 8, 4, 0, None, False),              # one token
    (5, 1000, 1352, 24, 4, 1, None, True),              # columns in no blocks, a last item of 72
    (16, 1024, 1408, 16, 4, 2, 1.0, False),             # 16 rows to an entry
    (64, 1032, 2176, 8, 2, 0, None, True),              # 32
    (64, 2056, 2176, 4, 3, 0, None, False),             # 64
])
def test_gated_layer_with_many_chunks(T, H, F, E, k, gating, cf, bias):
    """Large enough for the gate's and the up projection's chunks to alternate."""
    x, layer = make_layer(T + H, T, H, F, E, k, "swiglu", gating=gating, cf=cf, bias=bias)
    check_layer(x, layer)
    first = layer(x).clone()
    for _ in range(5):
        assert torch.equal(layer(x), first)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,H,F,E,k,act,gating,cf,bias", [
    (1, 128, 128, 1, 1, "gelu", 0, None, False),
    (1, 4096, 256, 8, 2, "swiglu", 0, None, False),
    (2, 384, 1408, 13, 3, "gelu", 1, None, True),       # chunks that end inside a K tile
    (9, 128, 640, 64, 4, "swiglu", 2, 0.8, True),
    (16, 1152, 256, 6, 2, "gelu", 0, None, False),
    (31, 256, 384, 3, 2, "swiglu", 0, None, False),
    (64, 256, 128, 4, 2, "gelu", 0, None, False),
])
def test_q4_layer_against_the_definition(group, T, H, F, E, k, act, gating, cf, bias):
    check_layer(*make_layer(T + H + E + group, T, H, F, E, k, act, gating, cf, bias, group))


@pytest.mark.parametrize("group", [0, 128])
def test_layer_at_the_decode_workloads_width(group):
    check_layer(*make_layer(7, 2, 4096, 14336, 3, 2, "gelu", group=group))


@pytest.mark.parametrize("T", [1, 2, 7, 32, 64])
def test_routing_is_that_of_the_whole_forward(T):
    """ids, weights, dispatch as moe_forward gives them, y within two
    roundings of its y."""
    x, layer = make_layer(T, T, 512, 256, 16, 4, bias=True, cf=1.1)
    y = layer(x)
    r = layer.routing
    full = moe.MoELayer(layer.w_router, layer.w1, layer.w2, 4, bias=layer.bias, capacity_factor=1.1)
    want = full(x)
    for n in ("ids", "counts", "offsets", "slot", "perm"):
        assert torch.equal(getattr(r, n), getattr(full.routing, n)), n
    torch.testing.assert_close(r.weights, full.routing.weights, rtol=0, atol=1e-5)
    rel = float((y.double() - want.double()).norm() / want.double().norm())
    # each side: h, y, and moe_forward's expert outputs rounded to bf16 (2^-8 at most each)
    assert rel <= 5 * 2.0 ** -8


def test_duplicate_router_columns_tie_to_the_lower_index():
    x, layer = make_layer(11, 6, 128, 64, 8, 3)
    w = layer.w_router.clone()
    w[:, 5] = w[:, 2]
    w[:, 7] = w[:, 2]
    tied = moe.MoEDecodeLayer(w, layer.w1, layer.w2, 8)
    tied(x)
    for row in tied.routing.ids.tolist():
        assert row.index(2) + 1 == row.index(5) and row.index(5) + 1 == row.index(7)


def test_masked_and_huge_biases():
    """Experts biased to -inf (or the lowest float) are chosen last, in index
    order, with weight 0; a token whose logits are all -inf still routes."""
    x, layer = make_layer(12, 4, 128, 64, 6, 3)
    bias = torch.zeros(6)
    bias[0], bias[2], bias[4], bias[5] = -math.inf, -math.inf, torch.finfo(torch.float32).min, -math.inf
    m = moe.MoEDecodeLayer(layer.w_router, layer.w1, layer.w2, 3, bias=bias.to(DEV))
    y = m(x)
    r = m.routing
    assert (r.ids[:, 2] == 4).all() and (r.weights[:, 2] == 0).all() and torch.isfinite(y).all()
    assert set(r.ids[:, :2].flatten().tolist()) == {1, 3}


@pytest.mark.parametrize("group", [0, 64])
def test_nan_and_inf_stay_in_their_token(group):
    x, layer = make_layer(13, 5, 256, 128, 4, 2, group=group)
    clean = layer(x).clone()
    bad = x.clone()
    bad[1, 17] = math.nan
    bad[3, 40] = math.inf
    y = layer(bad)
    assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any()


def test_everything_dropped_gives_zero_and_an_empty_batch_clears():
    x, layer = make_layer(14, 6, 128, 64, 8, 2, cf=1e-12)
    layer(x)
    torch.empty_like(x).fill_(7.0)
    y = layer(x)
    assert torch.equal(y, torch.zeros_like(y)) and layer.routing.counts.sum() == 0
    assert (layer.routing.slot == -1).all() and (layer.routing.perm == -1).all()
    y = layer(x[:0])
    assert y.shape == (0, 128)
    assert layer.routing.counts.tolist() == [0] * 8 and layer.routing.offsets.tolist() == [0] * 9
    assert moe.moe_get_device_status(layer.ws) == 0


def test_tokens_whose_rows_were_all_dropped_are_zero():
    x, layer = make_layer(15, 40, 128, 64, 4, 1, cf=0.3)
    y = check_layer(x, layer)
    dropped = (layer.routing.slot < 0).all(1)
    assert dropped.any() and (y[dropped] == 0).all()


def test_weights_past_32_bit_offsets():
    """Experts whose elements lie beyond 2^31 of the weight tensors."""
    E, H, F = 300 // 4, 2048, 16384
    w1 = torch.zeros(E, H, F, dtype=BF, device=DEV)   # 2.5e9 elements
    w2 = torch.zeros(E, F, H, dtype=BF, device=DEV)
    g = gen(16)
    last = E - 1
    w1[last] = randn(g, H, F, std=H ** -0.5).to(DEV)
    w2[last] = randn(g, F, H, std=F ** -0.5).to(DEV)
    w1[0] = 1.0
    w2[0] = 1.0
    bias = torch.zeros(E)
    bias[last] = 100.0
    x = randn(g, 2, H).to(DEV)
    layer = moe.MoEDecodeLayer(randn(g, H, E, std=H ** -0.5).to(DEV), w1, w2, 1, bias=bias.to(DEV))
    check_layer(x, layer)


@pytest.mark.parametrize("group", [0, 32])
def test_same_inputs_same_bits(group):
    x, layer = make_layer(17, 23, 1024, 704, 16, 4, "swiglu", group=group)
    first = layer(x).clone()
    for _ in range(20):
        assert torch.equal(layer(x), first)


def test_rows_do_not_depend_on_the_batch():
    """A token's y is the same whichever tokens are with it, but for where the
    K sums are cut: within the bound of either."""
    x, layer = make_layer(18, 12, 512, 256, 4, 2)
    whole = layer(x).double()
    for t in (0, 5, 11):
        one = layer(x[t:t + 1]).double()
        assert float((one - whole[t]).norm() / one.norm()) <= 2 * 2.0 ** -8


# ------------------------------------------------------------------ matvec --

def check_matvec(x, w, group, offsets, y):
    rows = x.shape[0]
    xd = x.cpu().double()
    done = torch.zeros(rows, dtype=torch.bool)
    for i in range(len(offsets) - 1):
        a, b = offsets[i], offsets[i + 1]
        if b <= a:
            continue
        m = ref.q4_values(w.codes[i % w.E:i % w.E + 1], w.scales[i % w.E:i % w.E + 1], group)[0]
        want = xd[a:b] @ m
        err = (w.K + w.K // group) * ref.U_F32 * (xd[a:b].abs() @ m.abs())
        err = err + ref.U_BF16 * (want.abs() + err) + 1e-37
        d = (y[a:b].cpu().double() - want).abs()
        assert (d <= err).all(), f"segment {i}: {float((d / err).max())} times the bound"
        done[a:b] = True
    return done


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K,N,E,offsets", [
    (1, 128, 8, 1, [0, 1]),
    (1, 4096, 128, 1, [0, 1]),                      # one item, many CTAs
    (1, 1408, 2048, 1, [0, 1]),
    (5, 384, 136, 2, [0, 0, 5]),                    # an empty segment
    (8, 256, 4104, 3, [0, 3, 3, 8]),
    (9, 256, 72, 1, [0, 9]),
    (17, 640, 200, 4, [2, 5, 5, 16, 17]),           # starts behind row 0
    (40, 128, 264, 2, [0, 10, 20, 25, 30]),         # more segments than matrices, rows left over
    (200, 256, 136, 2, [0, 130, 200]),              # segments over several row blocks
    (512, 128, 64, 1, [0, 512]),
])
def test_matvec_against_the_definition(group, rows, K, N, E, offsets):
    g = gen(rows + K + N)
    w = random_q4(g, E, K, N, group)
    x = randn(g, rows, K).to(DEV)
    out = torch.full((rows, N), 3.0, dtype=BF, device=DEV)
    y = moe.matvec_q4(x, w, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=out)
    assert y is out
    done = check_matvec(x, w, group, offsets, y)
    assert (y[~done.to(DEV)] == 3.0).all()          # rows outside every segment stay


def test_matvec_without_offsets_and_with_bad_ones():
    g = gen(31)
    w = random_q4(g, 1, 256, 128, 64)
    x = randn(g, 12, 256).to(DEV)
    y = moe.matvec_q4(x, w)
    check_matvec(x, w, 64, [0, 12], y)
    # offsets out of range are clamped and never followed; a decreasing one is an empty segment
    out = torch.full((12, 128), 3.0, dtype=BF, device=DEV)
    moe.matvec_q4(x, w, torch.tensor([-5, 4, 2, 1000], dtype=torch.int32, device=DEV), out=out)
    assert torch.equal(out, y)                      # rows 0..3, none, rows 2..11
    empty = moe.matvec_q4(x[:0], w)
    assert empty.shape == (0, 128)


def test_matvec_nan_scale_and_inf_rows():
    g = gen(32)
    w = random_q4(g, 1, 128, 64, 32)
    x = randn(g, 3, 128).to(DEV)
    clean = moe.matvec_q4(x, w)
    w.scales[0, 1, 5] = math.nan
    y = moe.matvec_q4(x, w)
    cols = [c for c in range(64) if c != 5]
    assert torch.isnan(y[:, 5]).all() and torch.equal(y[:, cols], clean[:, cols])
    x[1, 3] = math.inf
    y = moe.matvec_q4(x, w)
    assert torch.equal(y[[0, 2]][:, cols], clean[[0, 2]][:, cols])


@pytest.mark.parametrize("group", [32, 64, 128])
def test_matvec_largest_and_smallest_scales(group):
    """Scales near the ends of bf16's range, with rows that bring the result
    back inside: nothing on the way overflows or vanishes."""
    g = gen(34)
    for scale, xs in ((2.0 ** 125, 2.0 ** -60), (2.0 ** -118, 2.0 ** 60)):
        w = random_q4(g, 1, 384, 72, group)
        w.scales.copy_((w.scales.double().sign() * scale).bfloat16())
        x = (randn(g, 5, 384).double() * xs).bfloat16().to(DEV)
        y = moe.matvec_q4(x, w)
        assert torch.isfinite(y).all() and (y != 0).any()
        check_matvec(x, w, group, [0, 5], y)


def test_matvec_past_32_bit_offsets():
    E, K, N = 150, 4096, 4096                        # 2.5e9 weights
    codes = torch.full((E, K // 8, N), -1, dtype=torch.int32, device=DEV)
    scales = torch.ones(E, K // 128, N, dtype=BF, device=DEV)
    g = gen(33)
    last = random_q4(g, 1, K, N, 128)
    codes[E - 1], scales[E - 1] = last.codes[0], last.scales[0]
    w = moe.Q4Weights(codes, scales)
    x = randn(g, 2, K).to(DEV)
    offsets = [0] * E + [2]
    check_matvec(x, w, 128, offsets, moe.matvec_q4(x, w, torch.tensor(offsets, dtype=torch.int32, device=DEV)))


# ------------------------------------------------------- quantise and back --

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("E,K,N", [(1, 128, 8), (3, 256, 72), (2, 384, 136), (1, 1408, 520)])
def test_quantize_is_the_definition_bit_for_bit(group, E, K, N):
    g = gen(E + K + N + group)
    w = randn(g, E, K, N)
    w[0, :, 0] = 0.0                                  # a group of zeros
    w[0, :group, 1] *= 2.0 ** -120                    # scales below 2^-100
    w[0, :group, 2] = torch.tensor(2.0 ** -133).to(BF)   # the smallest subnormal: scale 0
    w[0, :group, 3] = (torch.randint(0, 60, (group,), generator=g).float() * 2.0 ** -133).to(BF)
    w[0, :group, 4] = torch.finfo(BF).max             # the largest: scale max / 7
    # every quotient a tie: multiples of half the scale
    w[0, :group, 5] = (torch.arange(group) % 15 - 7).float().to(BF) * 0.5
    w[0, 0, 5] = 7.0
    q = moe.quantize_q4(w.to(DEV), group)
    codes, scales = ref.quantize(w, group)
    assert torch.equal(q.scales.cpu().view(torch.int16), scales.view(torch.int16))
    assert torch.equal(ref.unpack_codes(q.codes), codes)
    # and back: the products rounded once
    want = ((codes - 8).double() * scales.double().repeat_interleave(group, 1)).to(BF)
    assert torch.equal(moe.dequantize_q4(q).cpu().double(), want.double())


def test_quantize_all_bf16_quotients():
    """Every |w| / scale that two bf16 mantissas can make in the top binades
    rounds as the exact quotient does."""
    m = torch.arange(128, 256)
    cols = []
    for mx in m.tolist():                             # max 1.0 .. 2.0: one scale each
        vals = torch.cat([m.float() / 128, m.float() / 256, m.float() / 512, -m.float() / 1024])
        vals = vals[vals.abs() <= mx / 128]
        col = torch.zeros(512)
        col[:vals.numel()] = vals
        col = col.view(4, 128)
        col[:, 127] = mx / 128                        # the largest of its group
        cols.append(col.reshape(-1))
    w = torch.stack(cols, 1).to(BF).unsqueeze(0)      # [1, 512, 128]
    q = moe.quantize_q4(w.to(DEV), 128)
    codes, scales = ref.quantize(w, 128)
    assert torch.equal(ref.unpack_codes(q.codes), codes) and torch.equal(q.scales.cpu(), scales)


def test_quantize_marks_nan_and_inf():
    w = torch.ones(1, 64, 8, dtype=BF)
    w[0, 3, 1] = math.nan
    w[0, 40, 2] = -math.inf
    q = moe.quantize_q4(w.to(DEV), 32)
    s = q.scales.cpu()
    assert torch.isnan(s[0, 0, 1]) and s[0, 1, 2] == math.inf
    back = moe.dequantize_q4(q).cpu()
    assert torch.isnan(back[0, :32, 1]).all() and not torch.isfinite(back[0, 32:, 2]).any()
    assert torch.isfinite(back[0, 32:, 1]).all() and torch.isfinite(back[0, :32, 2]).all()


def test_dequantize_any_codes_and_scales():
    g = gen(41)
    w = random_q4(g, 3, 128, 40, 32)
    w.scales[1, 2, 7] = torch.tensor(2.0 ** -133).to(BF)   # subnormal products
    w.scales[2, 0, 9] = torch.finfo(BF).max                # products that overflow
    want = ref.q4_values(w.codes, w.scales, 32).float().to(BF)
    assert torch.equal(moe.dequantize_q4(w).cpu().double(), want.double())


# ------------------------------------------------- streams, graphs, together --

@pytest.mark.parametrize("group", [0, 64])
def test_captured_and_replayed_with_new_inputs(group):
    x, layer = make_layer(51, 6, 512, 384, 8, 2, group=group)
    a, b = x.clone(), torch.randn_like(x)
    want_a, want_b = layer(a).clone(), layer(b).clone()
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(static)
        z = layer(y)                                  # a second call of the same capture
    want_za, want_zb = layer(want_a).clone(), layer(want_b).clone()
    for src, wy, wz in ((a, want_a, want_za), (b, want_b, want_zb), (a, want_a, want_za)):
        static.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(z, wz)


def test_two_graphs_and_an_eager_call_at_once():
    x, layer = make_layer(52, 4, 1024, 512, 8, 2)
    q = random_q4(gen(5), 1, 1024, 512, 64)
    xs = [torch.randn_like(x) for _ in range(3)]
    wants = [layer(v).clone() for v in xs]
    mv = moe.matvec_q4(xs[2], q).clone()
    graphs, ys = [], []
    for v in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(layer(v))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            e, m = layer(xs[2]), moe.matvec_q4(xs[2], q)
    torch.cuda.synchronize()
    for got, want in zip(ys + [e, m], wants + [mv]):
        assert torch.equal(got, want)


def test_stream_argument():
    x, layer = make_layer(53, 3, 256, 256, 8, 2)
    want = layer(x).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = layer(x, stream=s)
    z = layer(x, stream=s.cuda_stream)
    q = moe.quantize_q4(torch.randn(128, 64, device=DEV, dtype=torch.float32).to(BF), 32, stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want) and q.K == 128


def test_results_of_earlier_calls_stay():
    x, layer = make_layer(54, 2, 128, 64, 4, 2)
    y1 = layer(x)
    keep = y1.clone()
    layer(torch.randn_like(x))
    assert torch.equal(y1, keep)


@pytest.mark.parametrize("group", [0, 64])
def test_batches_of_changing_size_share_a_streams_workspace(group):
    _, layer = make_layer(56, 1, 256, 128, 8, 2, group=group)
    g = gen(57)
    for T in (2, 64, 2, 5, 64):
        check_layer(randn(g, T, 256).to(DEV), layer)
        if T == 64:
            large = layer.ws
    check_layer(randn(g, 1, 256).to(DEV), layer)
    assert layer.ws is large


def test_host_threads_on_one_stream():
    """Calls of several host threads land on the default stream, each with its
    two kernels together."""
    x, layer = make_layer(58, 6, 512, 256, 8, 2)
    q = random_q4(gen(59), 1, 512, 256, 32)
    xs = [torch.randn_like(x) for _ in range(4)]
    wants = [(layer(v).clone(), moe.matvec_q4(v, q).clone()) for v in xs]
    bad = []

    def work(v, want):
        for _ in range(50):
            got = layer(v), moe.matvec_q4(v, q)
            if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                bad.append(v)

    threads = [threading.Thread(target=work, args=a) for a in zip(xs, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("group", [0, 64])
def test_copies_and_replaced_tensors(group):
    """A copied layer works on its own memory; a weight whose tensor is given
    other memory stays what it was for the layer."""
    x, layer = make_layer(60, 3, 256, 128, 4, 2, group=group)
    want = layer(x).clone()
    twin = copy.deepcopy(layer)
    if group:
        layer.w1.scales.zero_()
    else:
        layer.w1.zero_()
    assert torch.equal(twin(x), want) and not torch.equal(layer(x), want)
    want = layer(x).clone()
    for t in (layer.w1.codes, layer.w1.scales) if group else (layer.w1,):
        t.data = torch.zeros_like(t)
    torch.cuda.empty_cache()
    assert torch.equal(layer(x), want)
    if group:                                        # the weights by themselves are refused
        with pytest.raises(ValueError, match="other memory"):
            moe.dequantize_q4(layer.w1)
        seg = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
        with pytest.raises(ValueError, match="other memory"):
            moe.matvec_q4(x, layer.w1, seg)


def test_wrong_device_types_and_strides_are_refused():
    x, layer = make_layer(55, 4, 128, 64, 4, 2)
    for bad in (x.float(), x.cpu(), x[:, :64], x.t().contiguous().t(), x[None]):
        with pytest.raises((ValueError, TypeError)):
            layer(bad)
    with pytest.raises(moe.MoEError):
        layer(torch.zeros(65, 128, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        moe.matvec_q4(x, random_q4(gen(6), 2, 128, 64, 32))    # two matrices, no offsets


def test_quantised_model_from_bf16_weights_to_prompt_and_decode():
    """The operators as they are used together: a bf16 layer quantised once,
    decoded with its 4-bit weights step by step, and a prompt run on the bf16
    matrices that the 4-bit ones stand for."""
    x, layer = make_layer(61, 20, 256, 384, 8, 2, "swiglu", bias=True)
    q1, q2 = moe.quantize_q4(layer.w1, 64), moe.quantize_q4(layer.w2, 64)
    small = moe.MoEDecodeLayer(layer.w_router, q1, q2, 2, bias=layer.bias, act="swiglu")
    prompt = moe.MoELayer(layer.w_router, moe.dequantize_q4(q1), moe.dequantize_q4(q2), 2, bias=layer.bias,
                          act="swiglu")
    want = prompt(x).double()
    step = torch.cat([small(x[t:t + 1]) for t in range(20)]).double()
    check_layer(x, small)
    # dequantised weights, h, expert outputs and y rounded to bf16 on one side, h and y on the other
    assert float((step - want).norm() / want.norm()) <= 6 * 2.0 ** -8
    # the same rows through the products one by one: h and y of expert 0
    r = small.routing
    xp = torch.empty(40, 256, dtype=BF, device=DEV)
    s = moe.make_shape(20, 256, 384, 8, 2, act="swiglu")
    moe.moe_dispatch_rows(s, x, r.perm, r.offsets, xp)
    z = moe.matvec_q4(xp, q1, r.offsets).float()
    h = (torch.nn.functional.silu(z[:, :384]) * z[:, 384:]).to(BF)
    Y = moe.matvec_q4(h, q2, r.offsets)
    y = torch.empty_like(x)
    moe.moe_combine(s, Y, r.weights, r.slot, y)
    whole = small(x).double()
    assert float((y.double() - whole).norm() / whole.norm()) <= 6 * 2.0 ** -8
    # quantising to 4 bits moves the layer's output by a quarter at most: 1/7 / sqrt(12) of the
    # largest weight per matrix, about 0.1 of a normal weight's size for each of three matrices
    assert float((layer(x).double() - whole).norm() / whole.norm()) <= 0.35

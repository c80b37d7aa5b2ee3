"""The decode operators on the GPU where other tests do not go: batches whose
cluster ranks have no rows of H, waits that run out, offsets that decrease,
rows whose mask leaves few experts or none, the calls by their C names."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

import decode_reference as ref
import mixture_experts_layer_12_gb300 as moe
from test_decode_gpu import (BF, DEV, check_layer, check_matvec, check_routing, gen, make_layer, random_q4,
                             randn)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_12_gb300 import build
    build.build()
    moe.load_library()


@pytest.mark.parametrize("H", [8, 16, 64, 120])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (8, 40, 3), (9, 4, 2), (64, 256, 8)])
def test_ranks_without_rows_of_h(H, T, E, k):
    """H is dealt to the 8 ranks in multiples of 16: some or most have none
    and reach the exchange of the partial logits long before the others."""
    x, layer = make_layer(H + T + E, T, H, 64, E, k)
    first = check_layer(x, layer).clone()
    ids = layer.routing.ids.clone()
    for _ in range(50):
        y = layer(x)
        assert torch.equal(y, first) and torch.equal(layer.routing.ids, ids)


@pytest.mark.parametrize("limit_ns", [2_000_000, 1000])
@pytest.mark.parametrize("T,H,F,E,k,act,group", [
    (1, 256, 256, 8, 2, "gelu", 0),          # h read by whoever needs it
    (16, 4096, 4096, 4, 1, "gelu", 0),       # h copied, shared items by their first CTA
    (64, 4096, 4096, 4, 2, "gelu", 0),       # h copied, shared items by all CTAs
    (16, 1024, 1408, 16, 4, "swiglu", 0),    # gate's and up projection's chunks in turn
    (1, 512, 768, 8, 2, "swiglu", 128),
    (6, 4096, 4096, 8, 2, "gelu", 64),
    (64, 2048, 2048, 4, 2, "swiglu", 32),    # two stages, one per consumer group
])
def test_waits_that_run_out(T, H, F, E, k, act, group, limit_ns):
    """Every CTA gives up and leaves, the status says so, the routing is the
    layer's, and the next call with the same workspace is right.  With 1 us
    the waits for the weights run out too."""
    x, layer = make_layer(T + H + F, T, H, F, E, k, act, group=group)
    want = check_layer(x, layer).clone()
    r, ws = layer.routing, layer.ws
    s = moe.make_shape(T, H, F, E, k, act=act)
    for t in (r.ids, r.weights, r.counts, r.offsets, r.perm, r.slot):
        t.zero_()
    y = torch.empty_like(x)
    for _ in range(3):
        moe.moed_selftest_wait_timeout(s, x, layer.w_router, None, layer.w1, layer.w2, y, r.ids, r.weights,
                                       r.counts, r.offsets, r.perm, r.slot, ws, limit_ns)
        with pytest.raises(moe.MoEError) as e:
            moe.moe_get_device_status(ws)
        assert e.value.code == moe.MOE_ERR_TIMEOUT
        check_routing(x, layer, r)
        for _ in range(2):
            assert torch.equal(layer(x), want)
            assert layer.ws is ws and moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("rows,n_segments,E", [(12, 3, 3), (100, 33, 5), (512, 256, 7), (37, 100, 64), (512, 40, 3)])
def test_matvec_decreasing_offsets_give_disjoint_segments(rows, n_segments, E):
    """Offsets against the contract: every row is computed once, by the first
    segment that reaches it, and rows that none reaches stay."""
    w = random_q4(gen(rows + E), E, 256, 136, 64)
    x = randn(gen(rows), rows, 256).to(DEV)
    rng = random.Random(rows + n_segments)
    for offsets in ([-5, 4, 2, 1000][:n_segments + 1] + [0, rows] * n_segments,
                    [rng.randint(-20, rows + 20) for _ in range(n_segments + 1)],
                    [rows // 3 + rng.randint(-2, 2) + i * rows // (2 * n_segments) for i in range(n_segments + 1)],
                    [rows] + [0] * n_segments):
        offsets = offsets[:n_segments + 1]
        rising = [max(min(max(o, 0), rows) for o in offsets[:i + 1]) for i in range(n_segments + 1)]
        out = torch.full((rows, 136), 3.0, dtype=BF, device=DEV)
        moe.matvec_q4(x, w, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=out)
        done = check_matvec(x, w, 64, rising, out)
        assert done.tolist() == [rising[0] <= r < rising[-1] for r in range(rows)]
        assert (out[~done.to(DEV)] == 3.0).all()


def masked_layer(T, E, k, gating, bias, group=0):
    x, layer = make_layer(T + E + k, T, 128, 64, E, k, gating=gating, group=group)
    return x, moe.MoEDecodeLayer(layer.w_router, layer.w1, layer.w2, k, bias=bias.to(DEV), gating=gating)


def same_as_forward(x, layer):
    """The routing, NaN included, is that of moe_forward."""
    full = moe.MoELayer(layer.w_router, layer.w1, layer.w2, layer.k, bias=layer.bias, gating=layer.gating)
    want = full(x)
    r, f = layer.routing, full.routing
    for n in ("ids", "counts", "offsets", "slot", "perm"):
        assert torch.equal(getattr(r, n), getattr(f, n)), n
    torch.testing.assert_close(r.weights, f.weights, rtol=0, atol=1e-5, equal_nan=True)
    return want


@pytest.mark.parametrize("gating", [0, 1, 2])
@pytest.mark.parametrize("T,E,k,allowed", [(1, 8, 4, [3]), (5, 40, 8, [39, 7]), (9, 8, 8, [1, 2, 5]), (64, 6, 5, [4])])
def test_more_choices_than_experts_that_are_not_masked(T, E, k, allowed, gating):
    """Masked experts come last, in index order and with weight 0."""
    bias = torch.full((E,), -math.inf)
    bias[allowed] = 0.0
    x, layer = masked_layer(T, E, k, gating, bias)
    y = layer(x)
    r = layer.routing
    n = len(allowed)
    masked = [e for e in range(E) if e not in allowed][:k - n]
    for row in r.ids.tolist():
        assert sorted(row[:n]) == sorted(allowed) and row[n:] == masked
    assert (r.weights[:, n:] == 0).all() and ((r.weights[:, :n].sum(1) - 1).abs() <= 1e-5).all()
    same_as_forward(x, layer)
    # the sum over the allowed experts alone: masked ones add 0 times a finite row
    ids = r.ids.cpu().long()
    lg, _, _ = ref.route(x, layer.w_router, layer.bias, k, gating)
    want, err = ref.experts(x, lambda e: layer.w1[e].cpu().double(), lambda e: layer.w2[e].cpu().double(), ids,
                            ref.gate(lg, ids, gating), r.slot.cpu(), "gelu")
    assert ((y.cpu().double() - want).abs() <= err).all()


@pytest.mark.parametrize("gating", [0, 1, 2])
@pytest.mark.parametrize("T,E,k,group", [(1, 8, 4, 0), (7, 40, 2, 32), (64, 6, 6, 0), (33, 16, 1, 64)])
def test_no_expert_left(T, E, k, group, gating):
    """Every expert masked: experts 0..k-1, a valid dispatch, NaN weights and y."""
    x, layer = masked_layer(T, E, k, gating, torch.full((E,), -math.inf), group)
    y = layer(x)
    r = layer.routing
    ids = torch.arange(k).expand(T, k)
    assert torch.equal(r.ids.cpu().long(), ids)
    assert torch.isnan(r.weights).all() and torch.isnan(y).all()
    for got, want in zip((r.counts, r.offsets, r.perm, r.slot), ref.dispatch(ids, E, T * k)):
        assert torch.equal(got.cpu(), want)
    assert moe.moe_get_device_status(layer.ws) == 0
    if not group:
        assert torch.isnan(same_as_forward(x, layer)).all()


@pytest.mark.parametrize("gating", [0, 1, 2])
def test_lowest_value_masks_are_no_infinities(gating):
    """Every expert at the type's lowest value: the logits round to it, all are
    equal, and the weights are those of equal logits."""
    low = torch.finfo(torch.float32).min
    x, layer = masked_layer(3, 8, 3, gating, torch.full((8,), low))
    y = layer(x)
    r = layer.routing
    assert r.ids.tolist() == [[0, 1, 2]] * 3
    want = 1 / 8 if gating == 1 else 1 / 3
    assert ((r.weights - want).abs() <= 1e-6).all() and torch.isfinite(y).all()
    same_as_forward(x, layer)


def buffers(layer, T):
    s = moe.make_shape(T, layer.H, layer.F, layer.E, layer.k, layer.capacity_factor, layer.gating, layer.act)
    r = moe.alloc_routing(T, layer.E, layer.k, DEV)
    ws = torch.empty(moe.moed_workspace_size(s), dtype=torch.uint8, device=DEV)
    return s, (r.ids, r.weights, r.counts, r.offsets, r.perm, r.slot), ws


@pytest.mark.parametrize("T,H,F,E,k,act,group", [
    (1, 256, 256, 8, 2, "gelu", 0), (40, 512, 384, 6, 3, "swiglu", 0), (16, 1024, 1408, 16, 4, "swiglu", 0),
    (9, 256, 640, 64, 4, "swiglu", 64), (64, 2048, 2048, 4, 2, "gelu", 32)])
def test_y_may_be_x(T, H, F, E, k, act, group):
    """moed_forward and moed_forward_q4 by name, written over their input, on
    another stream, eager and replayed."""
    x, layer = make_layer(T + H + E, T, H, F, E, k, act, bias=True, group=group)
    want = check_layer(x, layer).clone()
    s, r, ws = buffers(layer, T)
    fwd = moe.moed_forward_q4 if group else moe.moed_forward
    call = lambda v, st: fwd(s, v, layer.w_router, layer.bias, layer.w1, layer.w2, v, *r, ws, st)  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(st):
            v = x.clone()
        call(v, st)
        st.synchronize()
        assert torch.equal(v, want) and moe.moe_get_device_status(ws, st) == 0
    static, g = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call(static, st)
    for _ in range(3):
        static.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, want)
    for got, ref_ in zip(r, (layer.routing.ids, layer.routing.weights, layer.routing.counts, layer.routing.offsets,
                             layer.routing.perm, layer.routing.slot)):
        assert torch.equal(got, ref_)


def test_products_and_conversions_by_name():
    g = gen(71)
    w = randn(g, 3, 256, 72).to(DEV)
    q = moe.quantize_q4(w, 64)
    codes, scales = torch.empty_like(q.codes), torch.empty_like(q.scales)
    moe.moed_quantize_q4(w, codes, scales, 64)
    assert torch.equal(codes, q.codes) and torch.equal(scales.view(torch.int16), q.scales.view(torch.int16))
    out = torch.empty_like(w)
    moe.moed_dequantize_q4(q, out)
    assert torch.equal(out, moe.dequantize_q4(q))
    x = randn(g, 21, 256).to(DEV)
    offsets = [0, 4, 4, 21]
    seg = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y = torch.empty(21, 72, dtype=BF, device=DEV)
    ws = torch.empty(moe.moed_matvec_q4_workspace_size(21, 3, 256, 72), dtype=torch.uint8, device=DEV)
    moe.moed_matvec_q4(x, q, seg, y, ws)
    check_matvec(x, q, 64, offsets, y)
    assert torch.equal(y, moe.matvec_q4(x, q, seg)) and moe.moe_get_device_status(ws) == 0
    # no offsets: one segment of all rows, the first matrix
    with pytest.raises(moe.MoEError, match="moed_matvec_q4_workspace_size"):
        moe.moed_matvec_q4(x, q, None, y, ws)       # one segment of 21 rows needs more than three
    ws = torch.empty(moe.moed_matvec_q4_workspace_size(21, 1, 256, 72), dtype=torch.uint8, device=DEV)
    moe.moed_matvec_q4(x, q, None, y, ws)
    check_matvec(x, q, 64, [0, 21], y)


FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
import torch
import mixture_experts_layer_12_gb300 as moe
bf = dict(dtype=torch.bfloat16, device="cuda")
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") / 16).bfloat16()
w1, w2, wr = rnd(8, 256, 384), rnd(8, 384, 256), rnd(256, 8)
x = rnd(5, 256)
seg = torch.tensor([0, 1, 1, 2, 3, 3, 4, 4, 5], dtype=torch.int32, device="cuda")
layer = moe.MoEDecodeLayer(wr, w1, w2, 2)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = layer(x)
    none = layer(x[:0])
    q = moe.quantize_q4(w1, 64)
    back = moe.dequantize_q4(q)
    z = moe.matvec_q4(x, q, seg)
    z0 = moe.matvec_q4(x[:0], q, seg)
for _ in range(2):
    for t in (y, q.codes, q.scales, back, z):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    e = moe.quantize_q4(w1, 64)
    assert torch.equal(y, layer(x)) and torch.equal(q.codes, e.codes) and torch.equal(q.scales, e.scales)
    assert torch.equal(back, moe.dequantize_q4(e)) and torch.equal(z, moe.matvec_q4(x, e, seg))
    assert y.abs().sum() > 0 and z.abs().sum() > 0
print("ok")
"""


def test_a_process_whose_first_calls_are_captured():
    """Nothing of the library has run before the capture: kernels are loaded and
    set up inside it."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=ROOT)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]

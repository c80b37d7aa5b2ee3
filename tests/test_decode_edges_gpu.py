"""The decode operators on the GPU where other tests do not go: batches whose
cluster ranks have no rows of H, waits that run out, offsets that decrease."""
import random

import pytest
import torch

import mixture_experts_layer_12_gb300 as moe
from test_decode_gpu import (BF, DEV, check_layer, check_matvec, check_routing, gen, make_layer, random_q4,
                             randn)

pytestmark = pytest.mark.gpu


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

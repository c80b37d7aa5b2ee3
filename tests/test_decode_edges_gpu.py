"""The decode operators on the GPU where other tests do not go: batches whose
cluster ranks have no rows of H."""
import pytest
import torch

import mixture_experts_layer_12_gb300 as moe
from test_decode_gpu import check_layer, make_layer

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

"""Edges of embed, layer_norm, dispatch and combine: empty calls."""
import pytest
import torch

from test_layer_operators import nsp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1, 12_287, 12_288, 20_000])
def test_experts_of_no_tokens_with_many_choices(nsp, k):
    x = torch.zeros(0, 5, device="cuda")
    ids = torch.zeros(0, k, dtype=torch.int32, device="cuda")
    rows, order = nsp.dispatch(x, ids, 3)
    assert rows.shape == (0, 5) and order.place.shape == (0, k) and order.offsets.tolist() == [0] * 4
    assert nsp.combine(rows, order).shape == (0, 5)

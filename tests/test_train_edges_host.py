"""Host-side checks of the training operators at the limits of their sizes; no GPU."""
import pytest

from test_train_host import nsp  # noqa: F401


# ---- experts beyond the most ------------------------------------------------------
@pytest.mark.parametrize("N", [0, 10, 1 << 20, 2**32 - 1])
@pytest.mark.parametrize("E", [1025, 16384, 16385, 50257, 1 << 31, (1 << 31) + 8, 2**32 - 1])
def test_route_workspace_of_too_many_experts(nsp, N, E):
    """Logits of a vocabulary by mistake: no workspace (and an error from the call itself),
    where the layout's arithmetic divided by 0 or did not end."""
    assert nsp.ns_route_workspace(N, E) == 0


def test_route_workspace_up_to_the_most_experts(nsp):
    for E in (1, 8, 100, 512, 513, 1024):
        assert nsp.ns_route_workspace(1 << 20, E) % (8 * E + 4) == 0
        assert nsp.ns_route_workspace(1 << 20, E) > 0

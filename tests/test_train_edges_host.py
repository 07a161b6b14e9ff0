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


# ---- sizes that 32 bits do not hold ---------------------------------------------------
@pytest.mark.parametrize("size", [2**32, 2**32 + 4, 2**40, 2**63, -1])
def test_sizes_past_32_bits_are_refused(nsp, size):
    """What is left of them in 32 bits is another size, 4 for 2**32 + 4."""
    L = nsp._lib
    scan = [None, None, 0, 0, 0, 0, None, None, None, 1, 1, 1, 0]
    distill = [None, 1, None, None, None, None, None, 1, 1, 1, 0, 0, 0, 1.0]
    route = [None, 1, None, 1, 1, 1, 0, 0]
    calls = [lambda: nsp.ns_scan_workspace(size, 1, 1), lambda: nsp.ns_scan_workspace(1, size, 1),
             lambda: nsp.ns_scan_workspace(1, 1, size), lambda: nsp.ns_route_workspace(size, 1),
             lambda: nsp.ns_route_workspace(1, size)]
    for make, good, first in ((L.ns_scan_inputs, scan, 9), (L.ns_distill_inputs, distill, 7),
                              (L.ns_route_inputs, route, 3)):
        made = make(*good)
        for i in range(first, first + 3):
            assert getattr(made, make._fields_[i][0]) == 1
            bad = list(good)
            bad[i] = size
            calls.append(lambda make=make, bad=bad: make(*bad))
            last = make(*good[:i], 2**32 - 1, *good[i + 1:])
            assert getattr(last, make._fields_[i][0]) == 2**32 - 1
    for call in calls:
        with pytest.raises(nsp.NsPackError) as e:
            call()
        assert e.value.code == nsp.NS_ERR_INVALID_ARG


# ---- forward-mode derivatives -----------------------------------------------------------
def test_forward_mode_derivatives_are_refused(nsp):
    """They are refused before anything else is looked at (host tensors here)."""
    import torch
    import torch.autograd.forward_ad as forward_ad
    z, x = torch.randn(2, 5, 8), torch.randn(6, 40)
    top, ids = x.topk(3, 1)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        for call in (lambda: nsp.gated_scan(dual(z), z), lambda: nsp.gated_scan(z, dual(z)),
                     lambda: nsp.gated_scan(z, z, h0=dual(z[:, 0])),
                     lambda: nsp.distill_loss(dual(x), top, ids),
                     lambda: nsp.distill_loss(x, dual(top), ids), lambda: nsp.route(dual(x), 4)):
            with pytest.raises(NotImplementedError):
                call()
        with pytest.raises(nsp.NsPackError):  # no tangent: the device is what is wrong
            nsp.gated_scan(z, z)

"""Host-side checks of the training operators' C ABI that need no GPU: every
bad argument is refused before anything is enqueued.  Host addresses stand in
for device ones: each check below fails before their use."""
import ctypes as C

import numpy as np
import pytest


@pytest.fixture(scope="module")
def nsp():
    import __graft_entry__
    __graft_entry__.build()
    import deterministic_packed_assembly_gb300 as m
    return m


BUF = np.zeros(1 << 16, np.uint8)
AT = (BUF.ctypes.data + 255) & ~255


def scan(nsp, **kw):
    v = dict(z=AT, f=AT, z_row=80, z_time=8, f_row=80, f_time=8, bias=None, pos=None, doc=None, B=2,
             T=10, D=8, dtype=nsp.NS_F32)
    call = dict(h0=None, y=AT, h_last=AT, states=None)
    back = dict(states=AT, dy=AT, dy_row=80, dy_time=8, dh_last=None, dz=AT, df=AT, dbias=AT, dh0=AT,
                workspace=AT)
    for k, x in kw.items():
        (v if k in v else back if k.startswith("back_") else call)[k.replace("back_", "")] = x
    s = nsp._lib.ns_scan_inputs(*v.values())
    if any(k.startswith("back_") for k in kw):
        return lambda: nsp.ns_scan_backward(s, *back.values(), None)
    return lambda: nsp.ns_scan_forward(s, *call.values(), None)


def refused(nsp, call):
    with pytest.raises(nsp.NsPackError) as e:
        call()
    assert e.value.code == nsp.NS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(z=None), dict(f=None), dict(z=AT + 1), dict(f=AT + 2), dict(dtype=3), dict(dtype=-1),
    dict(z_row=-8), dict(f_time=-1), dict(z_time=1 << 50), dict(B=1 << 31), dict(T=1 << 31),
    dict(D=1 << 31), dict(B=1 << 20, D=1 << 16), dict(bias=AT + 2), dict(pos=AT + 1),
    dict(doc=AT + 3), dict(y=None), dict(y=AT + 1), dict(h_last=None), dict(h_last=AT + 2),
    dict(h0=AT + 1), dict(states=AT + 2),
    dict(back_states=None), dict(back_dy=None), dict(back_dz=None), dict(back_df=None),
    dict(back_dz=AT + 2), dict(back_dy_row=-1), dict(back_dy_time=1 << 60), dict(back_dh_last=AT + 1),
    dict(back_workspace=None), dict(back_workspace=AT + 2), dict(back_dbias=AT + 1),
    dict(back_dh0=AT + 2)])
def test_scan_refuses(nsp, kw):
    refused(nsp, scan(nsp, **kw))


def test_scan_of_nothing_is_ok(nsp):
    scan(nsp, B=0)()
    scan(nsp, D=0)()


def distill(nsp, **kw):
    v = dict(logits=AT, logits_row=64, top_logits=AT, top_ids=AT, teacher_lse=None, mask=None,
             weight=None, N=2, V=64, K=4, dtype=nsp.NS_BF16, top_dtype=nsp.NS_F32, ids_64=0,
             temperature=1.0)
    call = dict(loss=AT, dlogits=AT + 4096, dlogits_row=64)
    for k, x in kw.items():
        (v if k in v else call)[k] = x
    s = nsp._lib.ns_distill_inputs(*v.values())
    return lambda: nsp.ns_distill(s, *call.values(), None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=AT + 1), dict(logits_row=63), dict(logits_row=-64),
    dict(top_logits=None), dict(top_logits=AT + 2), dict(top_ids=None), dict(top_ids=AT + 4, ids_64=1),
    dict(V=0), dict(V=1 << 21), dict(K=0), dict(K=1025), dict(V=780_000, logits_row=780_000, K=257), dict(N=1 << 28), dict(dtype=9),
    dict(top_dtype=5), dict(teacher_lse=AT + 1), dict(weight=AT + 2), dict(loss=None),
    dict(loss=AT + 1), dict(dlogits=AT + 4097), dict(dlogits_row=10), dict(dlogits=AT + 64),
    dict(dlogits=AT, dlogits_row=65), dict(temperature=0.0), dict(temperature=-2.0),
    dict(temperature=float("nan")), dict(temperature=float("inf")), dict(temperature=1e-39)])
def test_distill_refuses(nsp, kw):
    refused(nsp, distill(nsp, **kw))


def test_distill_of_nothing_is_ok(nsp):
    distill(nsp, N=0)()


def route(nsp, back=False, **kw):
    v = dict(logits=AT, logits_row=16, doc=None, N=4, E=16, k=2, dtype=nsp.NS_F32, normalize=1)
    call = dict(ids=AT, weights=AT, counts=AT, tokens=AT, loss=AT, workspace=AT)
    grad = dict(ids=AT, weights=AT, counts=AT, tokens=AT, d_weights=AT, d_loss=AT, dlogits=AT)
    for k, x in kw.items():
        (v if k in v else grad if back else call)[k] = x
    s = nsp._lib.ns_route_inputs(*v.values())
    if back:
        return lambda: nsp.ns_route_backward(s, *grad.values(), None)
    return lambda: nsp.ns_route_forward(s, *call.values(), None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=AT + 2), dict(logits_row=15), dict(doc=AT + 1), dict(E=0),
    dict(E=1025, logits_row=1025), dict(k=0), dict(k=17), dict(E=64, logits_row=64, k=33),
    dict(dtype=4), dict(N=1 << 30), dict(ids=None), dict(ids=AT + 1), dict(weights=None),
    dict(counts=None), dict(tokens=AT + 2), dict(loss=None), dict(workspace=None, N=4096), dict(workspace=AT + 2),
    dict(back=True, ids=None), dict(back=True, weights=AT + 1), dict(back=True, counts=None),
    dict(back=True, tokens=None), dict(back=True, d_weights=AT + 2), dict(back=True, d_loss=AT + 1),
    dict(back=True, dlogits=None), dict(back=True, dlogits=AT + 2)])
def test_route_refuses(nsp, kw):
    refused(nsp, route(nsp, **kw))


def test_route_backward_of_nothing_is_ok(nsp):
    route(nsp, back=True, N=0)()


def test_structures_match_the_header(nsp):
    # three 64-bit pointers or strides and so on, as a C compiler lays them out
    L = nsp._lib
    assert C.sizeof(L.ns_scan_inputs) == 9 * 8 + 4 * 4
    assert C.sizeof(L.ns_distill_inputs) == 7 * 8 + 7 * 4 + 4
    assert C.sizeof(L.ns_route_inputs) == 3 * 8 + 5 * 4 + 4


def test_workspaces(nsp):
    assert nsp.ns_scan_workspace(3, 5, 10) == 3 * 10 * 4
    assert nsp.ns_scan_workspace(0, 5, 10) == 0
    assert nsp.ns_scan_workspace(1, 32, 64) == 64 * 4
    assert nsp.ns_scan_workspace(1, 10_000, 64) == 8 * 64 * 4  # eight blocks share the row
    assert nsp.ns_route_workspace(0, 16) == 0 and nsp.ns_route_workspace(8, 16) == 0
    assert nsp.ns_route_workspace(1 << 20, 64) >= nsp.ns_route_workspace(64, 64)

"""Host-side checks of embed, layer_norm, dispatch and combine that need no GPU: every bad
argument is refused before anything is enqueued.  Host addresses stand in for device
ones: each check below fails before their use."""
import ctypes as C

import pytest

from test_train_host import AT, nsp, refused  # noqa: F401


def embed(nsp, back=False, **kw):
    v = dict(tokens=AT, doc=None, N=4, V=10, D=8, table_dtype=nsp.NS_F32, dtype=nsp.NS_BF16, ids_64=0,
             scale=1.0)
    call = dict(dy=AT, dy_row=8, dtable=AT, workspace=AT) if back else dict(table=AT, table_row=8, y=AT)
    for k, x in kw.items():
        (v if k in v else call)[k] = x
    s = nsp._lib.ns_embed_inputs(*v.values())
    f = nsp.ns_embed_backward if back else nsp.ns_embed_forward
    return lambda: f(s, *call.values(), None)


@pytest.mark.parametrize("kw", [
    dict(tokens=None), dict(tokens=AT + 2), dict(tokens=AT + 4, ids_64=1), dict(doc=AT + 1),
    dict(N=1 << 31), dict(V=1 << 31), dict(D=1 << 31), dict(N=1 << 30, D=1 << 12),
    dict(V=1 << 30, D=1 << 12, table_row=1 << 12), dict(table_dtype=3), dict(dtype=-1),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(table=None), dict(table=AT + 2),
    dict(table_row=7), dict(table_row=-8), dict(table_row=1 << 45), dict(y=None), dict(y=AT + 1),
    dict(back=True, dy=None), dict(back=True, dy=AT + 1), dict(back=True, dy_row=7),
    dict(back=True, dy_row=0), dict(back=True, dtable=None), dict(back=True, dtable=AT + 2),
    dict(back=True, workspace=None), dict(back=True, workspace=AT + 8), dict(back=True, tokens=None),
    dict(back=True, V=1 << 31), dict(back=True, V=(1 << 31) - 1, D=1 << 12, dy_row=1 << 12)])
def test_embed_refuses(nsp, kw):
    refused(nsp, embed(nsp, **kw))


def norm(nsp, back=False, **kw):
    v = dict(x=AT, x_row=8, weight=AT, bias=None, doc=None, N=4, D=8, dtype=nsp.NS_BF16,
             weight_dtype=nsp.NS_F32, eps=1e-5)
    call = dict(mean=AT, rstd=AT, dy=AT, dy_row=8, dx=AT, dweight=AT, dbias=AT, workspace=AT)
    if not back:
        call = dict(y=AT, mean=None, rstd=None)
    for k, x in kw.items():
        (v if k in v else call)[k] = x
    s = nsp._lib.ns_norm_inputs(*v.values())
    f = nsp.ns_norm_backward if back else nsp.ns_norm_forward
    return lambda: f(s, *call.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=AT + 1), dict(x_row=7), dict(x_row=-8), dict(weight=AT + 2),
    dict(bias=AT + 1), dict(doc=AT + 2), dict(N=1 << 31), dict(D=1 << 30, x_row=1 << 30), dict(D=0),
    dict(dtype=5), dict(weight_dtype=2), dict(weight_dtype=7), dict(eps=-1e-9),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None), dict(y=AT + 1), dict(mean=AT + 2),
    dict(rstd=AT + 1),
    dict(back=True, mean=None), dict(back=True, rstd=None), dict(back=True, dy=None),
    dict(back=True, dy_row=5), dict(back=True, dx=None), dict(back=True, dx=AT + 1),
    dict(back=True, dweight=AT + 2), dict(back=True, dbias=AT + 1), dict(back=True, workspace=None),
    dict(back=True, workspace=AT + 2), dict(back=True, x=None)])
def test_norm_refuses(nsp, kw):
    refused(nsp, norm(nsp, **kw))


def experts(nsp, call="dispatch", **kw):
    v = dict(N=4, k=2, E=3, D=8, dtype=nsp.NS_F32)
    args = dict(
        dispatch=dict(ids=AT, x=AT, x_row=8, place=AT, slots=AT, offsets=AT, rows=AT, workspace=None),
        combine=dict(place=AT, offsets=AT, weights=None, rows=AT, rows_row=8, out=AT),
        backward=dict(place=AT, offsets=AT, weights=AT, rows=AT, rows_row=8, d_out=AT, d_out_row=8,
                      d_rows=AT, d_weights=AT))[call]
    for k, x in kw.items():
        (v if k in v else args)[k] = x
    s = nsp._lib.ns_expert_sizes(*v.values())
    f = dict(dispatch=nsp.ns_dispatch, combine=nsp.ns_combine, backward=nsp.ns_combine_backward)[call]
    return lambda: f(s, *args.values(), None)


@pytest.mark.parametrize("kw", [
    dict(k=0), dict(E=0), dict(E=1025), dict(N=1 << 30), dict(N=1 << 20, k=1 << 11),
    dict(D=1 << 30, x_row=1 << 30), dict(N=1 << 24, k=64, D=1 << 12, x_row=1 << 12), dict(dtype=3),
    dict(ids=None), dict(ids=AT + 2), dict(x=None), dict(x=AT + 1), dict(x_row=7), dict(x_row=-8),
    dict(place=None), dict(place=AT + 1), dict(slots=None), dict(offsets=None), dict(offsets=AT + 2),
    dict(rows=None), dict(rows=AT + 2), dict(N=4096), dict(workspace=AT + 1, N=4096),
    dict(call="combine", place=None), dict(call="combine", offsets=None),
    dict(call="combine", weights=AT + 2), dict(call="combine", rows=None),
    dict(call="combine", rows_row=7), dict(call="combine", rows_row=0), dict(call="combine", out=None),
    dict(call="combine", out=AT + 2), dict(call="combine", E=0), dict(call="combine", dtype=9),
    dict(call="backward", place=None), dict(call="backward", offsets=AT + 1),
    dict(call="backward", rows=None), dict(call="backward", rows_row=4),
    dict(call="backward", d_out=None), dict(call="backward", d_out_row=7),
    dict(call="backward", d_rows=None), dict(call="backward", d_weights=AT + 2),
    dict(call="backward", weights=AT + 1)])
def test_experts_refuse(nsp, kw):
    refused(nsp, experts(nsp, **kw))


def test_calls_of_nothing_are_ok(nsp):
    embed(nsp, N=0, tokens=None, table=None, y=None)()
    embed(nsp, D=0, table_row=0)()
    embed(nsp, back=True, V=0)()
    norm(nsp, N=0, x=None, y=None)()
    experts(nsp, "combine", N=0)()
    experts(nsp, "combine", D=0, rows_row=0)()
    experts(nsp, "backward", N=0)()


def test_structures_match_the_header(nsp):
    L = nsp._lib
    assert C.sizeof(L.ns_embed_inputs) == 2 * 8 + 7 * 4 + 4
    assert C.sizeof(L.ns_norm_inputs) == 5 * 8 + 5 * 4 + 4
    assert C.sizeof(L.ns_expert_sizes) == 5 * 4


def test_workspaces(nsp):
    for N in (0, 1, 31, 32, 33, 5000, 1 << 20):
        for V in (1, 600, 200000):
            assert nsp.ns_embed_workspace(N, V, 40) >= 8 * N + V
    assert nsp.ns_embed_workspace(1 << 31, 5, 5) == 0 and nsp.ns_embed_workspace(5, 5, 1 << 31) == 0
    assert nsp.ns_norm_workspace(0, 64) == 0 and nsp.ns_norm_workspace(1, 64) == 2 * 64 * 4
    assert nsp.ns_norm_workspace(1 << 20, 9000) % (2 * 9000 * 4) == 0
    assert nsp.ns_dispatch_workspace(0, 2, 8) == 0 and nsp.ns_dispatch_workspace(64, 8, 64) == 0
    assert nsp.ns_dispatch_workspace(1 << 20, 2, 64) >= 65 * 4
    for bad in ((10, 0, 5), (10, 2, 0), (10, 2, 1025), (1 << 30, 2, 8)):
        assert nsp.ns_dispatch_workspace(*bad) == 0


@pytest.mark.parametrize("size", [2**32, 2**32 + 4, 2**63, -1])
def test_sizes_past_32_bits_are_refused(nsp, size):
    L = nsp._lib
    made = dict(ns_embed_inputs=([None, None, 1, 1, 1, 0, 0, 0, 1.0], (2, 3, 4)),
                ns_norm_inputs=([None, 1, None, None, None, 1, 1, 0, 0, 1e-5], (5, 6)),
                ns_expert_sizes=([1, 1, 1, 1, 0], (0, 1, 2, 3)))
    calls = [lambda: nsp.ns_embed_workspace(size, 1, 1), lambda: nsp.ns_embed_workspace(1, size, 1),
             lambda: nsp.ns_embed_workspace(1, 1, size), lambda: nsp.ns_norm_workspace(size, 1),
             lambda: nsp.ns_norm_workspace(1, size), lambda: nsp.ns_dispatch_workspace(size, 1, 1),
             lambda: nsp.ns_dispatch_workspace(1, size, 1), lambda: nsp.ns_dispatch_workspace(1, 1, size)]
    for name, (good, at) in made.items():
        make = getattr(L, name)
        make(*good)
        for i in at:
            bad = list(good)
            bad[i] = size
            calls.append(lambda make=make, bad=bad: make(*bad))
    for call in calls:
        refused(nsp, call)


def test_host_tensors_and_forward_mode_are_refused(nsp):
    import torch
    import torch.autograd.forward_ad as forward_ad
    x, ids = torch.randn(6, 8), torch.zeros(6, 2, dtype=torch.int32)
    order = nsp.ExpertOrder(ids, ids.view(-1), torch.zeros(4, dtype=torch.int32))
    for call in (lambda: nsp.embed(x, ids), lambda: nsp.embed_backward(x, ids[:, 0], 9),
                 lambda: nsp.embed_backward(x, ids[:, 0], 2**31), lambda: nsp.layer_norm(x),
                 lambda: nsp.dispatch(x, ids, 3), lambda: nsp.combine(torch.randn(12, 8), order)):
        refused(nsp, call)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        for call in (lambda: nsp.embed(dual(x), ids), lambda: nsp.layer_norm(dual(x)),
                     lambda: nsp.layer_norm(x, dual(x[0].clone())), lambda: nsp.dispatch(dual(x), ids, 3),
                     lambda: nsp.combine(dual(x), order), lambda: nsp.combine(x, order, dual(x))):
            with pytest.raises(NotImplementedError):
                call()

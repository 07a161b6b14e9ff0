"""Edges of embed, layer_norm, dispatch and combine: empty calls, the widths at which another
kernel takes over, and waits that run out."""
import pytest
import torch

from test_layer_operators import DTYPES, check_norm, gen, norm_inputs, nsp, same  # noqa: F401

pytestmark = pytest.mark.gpu

# where a shape of a row's threads ends (norm_shape), batches of the ring become smaller (floats
# and 16 bits in turn), and the ring ends: 17920 of 16 bits and 11520 floats backward, 19200 forward
BORDERS = (512, 768, 1280, 1536, 2560, 3328, 3840, 5120, 6400, 6656, 7680, 8960, 11520, 14080, 17920,
           19200)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [D + more for D in BORDERS for more in (0, 1)])
def test_layer_norm_at_the_widths_where_kernels_change(nsp, D, dtype):
    """Rows of the widths on both sides: with enough of them for the ring, the values, and the
    same bits as of a few (which forward go another way)."""
    x, w, b, doc, dy = norm_inputs(617, D, dtype, "f32", D)
    check_norm(nsp, x, w, b, doc, dy)
    x, w, b, doc, dy = (t.cuda() for t in (x, w, b, doc, dy))
    y, m, r = nsp.layer_norm_forward(x, w, b, doc=doc)
    dx = nsp.layer_norm_backward(dy, x, w, b, m, r, doc=doc)[0]
    n = slice(300, 303)
    y3, m3, r3 = nsp.layer_norm_forward(x[n], w, b, doc=doc[n])
    assert same(y3, y[n]) and same(m3, m[n]) and same(r3, r[n])
    assert same(nsp.layer_norm_backward(dy[n], x[n], w, b, m3, r3, doc=doc[n])[0], dx[n])


def wide_inputs(N, D, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + D)
    x, dy = (torch.randn(N, D, generator=g, device="cuda").to(DTYPES[dtype]) for _ in range(2))
    w, b = (torch.randn(D, generator=g, device="cuda") for _ in range(2))
    return x, dy, w, b


def probe(nsp, x, dy, w, b, doc, mean, rstd, fed, weights=True):
    """Outputs of both passes where only `fed` rows come; filled with 7 before."""
    from deterministic_packed_assembly_gb300.layers import _norm_inputs
    N, D = x.shape
    inputs = _norm_inputs(x, w, b, 1e-5, doc)
    stream = torch.cuda.current_stream().cuda_stream
    y, dx = torch.full_like(x, 7), torch.full_like(x, 7)
    m, r = torch.full_like(mean, 7), torch.full_like(rstd, 7)
    dw, db = torch.full_like(w, 7), torch.full_like(w, 7)
    work = torch.empty(nsp.ns_norm_workspace(N, D) // 4, device="cuda")
    nsp._lib.ns_norm_probe_forward(inputs, fed, y.data_ptr(), m.data_ptr(), r.data_ptr(),
                                   stream)
    nsp._lib.ns_norm_probe_backward(inputs, fed, mean.data_ptr(), rstd.data_ptr(),
                                    dy.data_ptr(), D, dx.data_ptr(),
                                    dw.data_ptr() if weights else None,
                                    db.data_ptr() if weights else None,
                                    work.data_ptr() if weights else None, stream)
    torch.cuda.synchronize()
    return y, m, r, dx, dw, db


@pytest.mark.parametrize("D,dtype,fed,weights", [
    (600, "bf16", 20_000, True), (2560, "bf16", 6000, False), (2571, "f16", 5000, True),
    (5003, "f32", 2400, True), (16384, "f16", 1600, True), (600, "bf16", 0, True)])
def test_a_wait_that_runs_out_shows_in_every_output(nsp, D, dtype, fed, weights):
    """Rows of which nothing comes: y, mean, rstd and dx of them all are NaN, padding among
    them, whatever their places in the ring held before (padding here, over some turns of
    it), and so are the weights' gradients; the other rows have their values."""
    N = fed + 1300
    x, dy, w, b = wide_inputs(N, D, dtype)
    doc = torch.zeros(N, dtype=torch.int32, device="cuda")
    doc[16:fed] = -1
    doc[fed + 2::3] = -1
    y, mean, rstd = nsp.layer_norm_forward(x, w, b, doc=doc)
    dx = nsp.layer_norm_backward(dy, x, w, b, mean, rstd, doc=doc)[0]
    want = y, mean, rstd, dx
    got = probe(nsp, x, dy, w, b, doc, mean, rstd, fed, weights)
    for a, e, name in zip(got, want, ("y", "mean", "rstd", "dx")):
        assert same(a[:fed], e[:fed]), name
        assert torch.isnan(a[fed:]).all(), (name, int((~torch.isnan(a[fed:])).sum()))
    for t in got[4:]:
        assert torch.isnan(t).all() if weights else (t == 7).all()
    # nothing of it is left
    assert all(same(a, e) for a, e in zip(probe(nsp, x, dy, w, b, doc, mean, rstd, N), want))


@pytest.mark.parametrize("k", [1, 12_287, 12_288, 20_000])
def test_experts_of_no_tokens_with_many_choices(nsp, k):
    x = torch.zeros(0, 5, device="cuda")
    ids = torch.zeros(0, k, dtype=torch.int32, device="cuda")
    rows, order = nsp.dispatch(x, ids, 3)
    assert rows.shape == (0, 5) and order.place.shape == (0, k) and order.offsets.tolist() == [0] * 4
    assert nsp.combine(rows, order).shape == (0, 5)


def chain(nsp, leaves, tokens, ids, doc, dy):
    """Loss and gradients of all four operators in a row."""
    table, w, b, gate = leaves
    x = nsp.layer_norm(nsp.embed(table, tokens, doc=doc), w, b, doc=doc)
    rows, order = nsp.dispatch(x, ids, 7)
    out = nsp.combine(torch.tanh(rows), order, gate)
    loss = (out.float() * dy).sum()
    return [loss.detach(), *torch.autograd.grad(loss, leaves)]


def chain_inputs(N, D, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    leaves = [t.requires_grad_() for t in (
        torch.randn(90, D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda"),
        torch.randn(D, generator=g, device="cuda"), torch.rand(N, 3, generator=g, device="cuda"))]
    tokens = torch.randint(0, 95, (N,), generator=g, device="cuda").int()
    ids = torch.randint(-1, 7, (N, 3), generator=g, device="cuda").int()
    doc = torch.randint(-1, 4, (N,), generator=g, device="cuda").int()
    return leaves, tokens, ids, doc, torch.randn(N, D, generator=g, device="cuda")


@pytest.mark.parametrize("N,D", [(60, 72), (3000, 640)])
def test_a_training_step_is_captured_in_a_graph(nsp, N, D):
    """Forward and backward through PyTorch's autograd, captured and replayed on new inputs."""
    args = chain_inputs(N, D, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(nsp, *args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(nsp, *args)
    for seed in (2, 3):
        new = chain_inputs(N, D, seed)
        with torch.no_grad():
            for a, b in zip([*args[0], *args[1:]], [*new[0], *new[1:]]):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, chain(nsp, *new)):
            assert same(a, b) or a.dim() == 0 and torch.allclose(a, b)


def test_calls_of_two_threads(nsp):
    """Two threads, a stream each: the bits of one alone."""
    import threading
    inputs = [chain_inputs(2000, 640, s) for s in (4, 5)]
    want = [chain(nsp, *i) for i in inputs]
    got = [[], []]

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[k].append(chain(nsp, *inputs[k]))
            torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert len(got[k]) == 20
        for g in got[k]:
            assert all(same(a, b) for a, b in zip(g[1:], want[k][1:]))

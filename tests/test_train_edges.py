"""The training operators at the edges of their definitions: a NaN gate where a
document starts, gates near 0 and near 1, logits of a type's lowest value, a NaN
teacher, forward-mode derivatives, states written over their input, sums of many
rows.  The references are those of test_train_operators, in 64 bits on the host.

Tolerances, with u = 2**-24, are derived at each test.
"""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from test_train_operators import (  # noqa: F401
    DTYPES, INF, NAN, ROUND, check_route, close, dev, distill_inputs, distill_reference, gen, nsp, refused,
    run_distill, scan_inputs, scan_reference)

pytestmark = pytest.mark.gpu

U = 2.0**-24


# ---- a document's NaN gate stays in the document --------------------------------
def starts_of(B, T):
    """Steps at which each row's second document starts: the first one, the middle, a
    segment of eight's edge, its last step, a tile of 64's edge, the last step."""
    at = [0, T // 2, T // 16 * 8, T // 16 * 8 + 7, T // 128 * 64, T - 1]
    return [min(at[b % len(at)], T - 1) for b in range(B)]


def check_nan_gates(nsp, B, T, D, dtype, shift=0):
    host, cuda, dy, dh = scan_inputs(B, T, D, dtype, B + T + D, packed=False, shift=shift)
    pos = torch.arange(1, T + 1).expand(B, T).clone().int()
    channels = [0, D // 2, D - 1]
    for b, s in enumerate(starts_of(B, T)):
        pos[b, s] = 0
        for k, c in enumerate(channels):
            host["f"][b, s, c] = (NAN, INF, NAN)[k]
    doc = torch.zeros(B, T, dtype=torch.int32)
    doc[:, T // 3] = -1  # padding between (where it is the start, the row has one document)
    host.update(pos=pos, doc=doc)
    cuda["f"].copy_(host["f"])
    want = scan_reference(**host, dy=dy, dh=dh)
    kw = dict(pos=pos.cuda(), doc=doc.cuda())
    bias, h0 = dev(host["bias"]), dev(host["h0"])
    y, h, states = nsp.gated_scan_forward(cuda["z"], cuda["f"], bias, h0=h0, **kw)
    got = nsp.gated_scan_backward(cuda["dy"], dev(dh), cuda["z"], cuda["f"], bias, states, **kw)
    for g, name in zip((y, h, *got), ("y", "h_last", "dz", "df", "dbias", "dh0")):
        floor = float(dy.double().abs().max()) if name in ("dbias", "dh0") else 0.0
        close(g, want[name], 2e-5, name, 0.0 if name in ("h_last", "dbias", "dh0") else ROUND[dtype],
              floor)
    # the documents before are what they are without the NaN
    assert not torch.isnan(want["dh0"]).any()
    for b, s in enumerate(starts_of(B, T)):
        assert not torch.isnan(got[0][b, :s]).any() and not torch.isnan(got[1][b, :s]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 130, 517, 1200])
def test_scan_nan_gate_where_a_document_starts(nsp, T, dtype):
    """With test_train_operators' tolerances: beside the NaN these are its inputs."""
    check_nan_gates(nsp, 6, T, 34, dtype)
    check_nan_gates(nsp, 6, T, 33, dtype, shift=1)


@pytest.mark.parametrize("T", [32, 100])
def test_scan_nan_gate_in_many_rows(nsp, T):
    # rows of a thread alone, and rows of a block alone
    check_nan_gates(nsp, 306, T, 130, "bf16")


# ---- gates near 0 -----------------------------------------------------------------
def gate_error(x, bias):
    """Bound of the relative error of both gates at x = f + bias: the exponent t = x log2 e is
    rounded by half a unit of |t|, and so is bias log2 e (ln 2 log2 e = 1), log2 e itself
    is off by 2**-26 of it; 2 units of 2**-23 from 2^t, 1 from 1/d, half a unit each from 1 + u and
    the product: 8 u."""
    return U * (1.25 * abs(x) + abs(bias) + 8)


@pytest.mark.parametrize("bias", [0.0, 3.0])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 40, 300])
@pytest.mark.parametrize("B,D", [(2, 17), (2, 18), (400, 130)])
def test_scan_closed_gates_keep_their_digits(nsp, B, D, T, bias):
    """A row that starts with a closed gate: dh0 = a_0 d_0 and the part a_0 h0 of the states
    (z = 0 there is nothing else) to the gate's own relative error, and 3 u for each product
    of the some 50 steps that are remembered."""
    x0 = torch.linspace(-20.0, -2.0, D)
    f = torch.full((B, T, D), 2.0) - bias
    f[:, 0] = x0 - bias
    z = torch.zeros(B, T, D)
    h0 = torch.rand(B, D, generator=gen(1)) + 0.5
    dy = torch.rand(B, T, D, generator=gen(2)) + 0.5
    b = torch.full((D,), bias)
    want = scan_reference(z, f, b, None, None, h0, dy=dy)
    y, h, st = nsp.gated_scan_forward(z.cuda(), f.cuda(), b.cuda(), h0=h0.cuda())
    _, _, _, dh0 = nsp.gated_scan_backward(dy.cuda(), None, z.cuda(), f.cuda(), b.cuda(), st)
    # the later steps' gates, at x = 2, add theirs as long as they are remembered
    bound = gate_error(20 + abs(bias), bias) + 3 * U * min(T, 50) + min(T, 50) * 0.14 * gate_error(2, bias)
    assert ((dh0.double().cpu() - want["dh0"]).abs() <= bound * want["dh0"]).all()
    first = (y[:, 0].double().cpu() - want["y"][:, 0]).abs()
    assert (first <= bound * want["y"][:, 0]).all()
    some = min(T, 30) - 1
    assert ((y[:, some].double().cpu() - want["y"][:, some]).abs() <= bound * want["y"][:, some]).all()


# ---- gates near 1 -------------------------------------------------------------------
@pytest.mark.parametrize("T,B,D", [(4096, 1, 8), (20_000, 1, 8), (20_000, 2, 33), (1000, 310, 4)])
def test_scan_long_memories(nsp, T, B, D):
    """Constant gates of x = 8 to 14, which are the same step after step, so that what each
    rounds the same way adds up.  Values are positive, so that a bound is relative.  From a
    state to the one 32 steps on the run's factor, just below 1, is rounded once (u / 2) and the
    state once (u): 1.5 u each 32 steps.  What the run adds, and how far its factor is from 1, is
    sums of 32 positive terms, off by 64 u and the gates' own error of themselves: such an error
    of c changes what is remembered by (1 + T c) times it."""
    g = gen(T + D)
    bias = torch.linspace(8.0, 14.0, D)
    f = torch.zeros(B, T, D)
    z = torch.rand(B, T, D, generator=g) + 0.5
    dy = torch.rand(B, T, D, generator=g) + 0.5
    h0 = torch.rand(B, D, generator=g) * 2 + 0.5
    dh = torch.rand(B, D, generator=g) + 0.5
    rows = slice(0, min(B, 2))  # the reference is slow
    want = scan_reference(z[rows], f[rows], bias, None, None, h0[rows], dy=dy[rows], dh=dh[rows])
    zc, fc, bc = z.cuda(), f.cuda(), bias.cuda()
    y, h, st = nsp.gated_scan_forward(zc, fc, bc, h0=h0.cuda())
    dz, df, _, dh0 = nsp.gated_scan_backward(dy.cuda(), dh.cuda(), zc, fc, bc, st)
    c = torch.sigmoid(-bias.double())
    gates = torch.tensor([gate_error(float(x), float(x)) for x in bias], dtype=torch.float64)
    bound = U * (1.5 * T / 32 + 64) + (1 + T * c) * (gates + 64 * U)

    def near(got, w, name, size=None):
        got = got.double().cpu()[rows]
        off = ((got - w).abs() / (bound * (w.abs() if size is None else size))).max()
        assert off <= 1, (name, float(off))

    near(y, want["y"], "y")
    near(h, want["h_last"], "h_last")
    near(dz, want["dz"], "dz")
    near(dh0, want["dh0"], "dh0")
    # df takes the difference of two values, of which each is as near as that
    before = torch.cat([h0[rows].double()[:, None], want["y"][:, :-1]], 1)
    near(df, want["df"], "df", (1 - c) * want["dz"] * (before + z[rows].double()))


# ---- distillation ----------------------------------------------------------------------
@pytest.mark.parametrize("temp", [0.25, 0.5, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 90_000])
def test_distill_teacher_chooses_a_masked_token(nsp, V, dtype, temp):
    """Logits of the type's lowest value at the teacher's choices: the loss is large, not a
    NaN.  It is a sum of terms of that size, of which each is rounded a few times: 2e-5 as
    elsewhere."""
    c = distill_inputs(4, V, 6, dtype, 5, temp=temp)
    low = torch.finfo(DTYPES[dtype]).min
    c["logits"][0, c["ids"][0, 0].long()] = low
    c["logits"][1, c["ids"][1, 3].long()] = low
    c["logits"][2, c["ids"][2].long()] = low
    c["top"][0, 0] += 1.0  # the first choice has most of the probability
    want_loss, want_g = distill_reference(**c)
    assert torch.isfinite(want_loss).all() and (want_loss[[0, 2]] > 1e35).all()
    loss, g = run_distill(nsp, c)
    assert ((loss.double().cpu() - want_loss).abs() <= 2e-5 * (1 + want_loss.abs())).all()
    assert torch.isfinite(g).all()
    scale = temp * c["weight"].double().abs()[:, None]
    assert ((g.double().cpu() - want_g).abs() <= 4e-5 * scale + ROUND[dtype] * 1.01 * want_g.abs()).all()


# ---- a NaN teacher
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [300, 90_000])
def test_distill_nan_teacher_makes_its_row_nan(nsp, V, tail):
    # m = sum p is a NaN, and m q with it at every place of the row
    c = distill_inputs(4, V, 6, "f32", 6, tail)
    want = run_distill(nsp, c)
    for at in (0, 4):
        d = dict(c, top=c["top"].clone())
        d["top"][2, at] = NAN
        loss, g = run_distill(nsp, d)
        assert torch.isnan(loss[2]) and torch.isnan(g[2]).all()
        for r in (0, 1, 3):
            assert torch.equal(loss[r], want[0][r]) and torch.equal(g[r], want[1][r])


# ---- forward-mode derivatives --------------------------------------------------------------
def test_forward_mode_derivatives_are_refused(nsp):
    """They are not there: an error, not outputs without a tangent."""
    z = torch.randn(2, 5, 8).cuda()
    x = torch.randn(6, 40).cuda()
    top, ids = x.topk(3, 1)
    h0, bias, lse = torch.zeros(2, 8).cuda(), torch.zeros(8).cuda(), torch.zeros(6).cuda() + 9
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        for call in (
                lambda: nsp.gated_scan(dual(z), z), lambda: nsp.gated_scan(z, dual(z)),
                lambda: nsp.gated_scan(z, z, dual(bias)), lambda: nsp.gated_scan(z, z, h0=dual(h0)),
                lambda: nsp.distill_loss(dual(x), top, ids),
                lambda: nsp.distill_loss(x, dual(top), ids),
                lambda: nsp.distill_loss(x, top, ids, teacher_lse=dual(lse)),
                lambda: nsp.route(dual(x), 4)):
            for grad in (True, False):
                with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError):
                    call()
        assert nsp.gated_scan(z, z)[0].shape == z.shape  # others of the level go on
        # the gradients of an output that are duals themselves
        zr, xr = z.clone().requires_grad_(), x.clone().requires_grad_()
        for y, at in ((nsp.gated_scan(zr, z)[0], zr), (nsp.distill_loss(xr, top, ids), xr),
                      (nsp.route(xr, 4).weights, xr)):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(y, at, dual(torch.ones_like(y)))


# ---- sizes past 32 bits -----------------------------------------------------------------------
def test_sizes_past_32_bits_are_refused(nsp):
    """Four more than 2**32: not four."""
    n = 2**32 + 4
    z = torch.zeros(1, 1, 1, dtype=torch.bfloat16, device="cuda").expand(1, n, 1)
    refused(nsp, lambda: nsp.gated_scan(z, z))
    x = torch.empty(n, 1, dtype=torch.bfloat16, device="cuda")
    refused(nsp, lambda: nsp.route(x, 1))
    top = torch.empty(n, 1, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    refused(nsp, lambda: nsp.distill_loss(x, top, ids))


# ---- states over their input --------------------------------------------------------------------
@pytest.mark.parametrize("T", [60, 100, 129, 200, 300, 400, 500, 512, 513, 2000])
def test_scan_last_states_over_the_first(nsp, T):
    # h_last may be h0: in clusters of every size, of one round and of several
    host, cuda, _, _ = scan_inputs(2, T, 96, "f32", T, packed=False)
    h0, bias = dev(host["h0"]), dev(host["bias"])
    want = nsp.gated_scan(cuda["z"], cuda["f"], bias, h0=h0)
    for _ in range(5):
        h, y = h0.clone(), torch.empty_like(want[0])
        inputs = nsp._lib.ns_scan_inputs(
            cuda["z"].data_ptr(), cuda["f"].data_ptr(), T * 96, 96, T * 96, 96, bias.data_ptr(), None,
            None, 2, T, 96, nsp.NS_F32)
        nsp.ns_scan_forward(inputs, h.data_ptr(), y.data_ptr(), h.data_ptr(), None,
                            torch.cuda.current_stream().cuda_stream)
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


# ---- the bias's gradient ---------------------------------------------------------------------------
def dirty_memory():
    """What PyTorch hands out next holds NaN."""
    junk = [torch.full((n,), NAN, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24)]
    del junk


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(60, 700, 355), (64, 200, 320), (2, 300, 64), (310, 70, 33), (60, 24, 1300)])
def test_scan_bias_gradient_of_many_rows(nsp, B, T, D, dtype):
    """Blocks with whole rows and clusters beside them share a workspace, some rows of which
    are zeros.  dbias against the sum, in 64 bits, of the df that came with it: in 16 bits
    each of those is off by its own rounding.  A term goes through at most T / 8 additions in
    its warp, 8 between warps and B + 8 between rows, each off by u of at most the sizes' sum."""
    host, cuda, dy, dh = scan_inputs(B, T, D, dtype, B + T)
    kw = dict(pos=dev(host["pos"]), doc=dev(host["doc"]))
    bias, h0 = dev(host["bias"]), dev(host["h0"])
    _, _, st = nsp.gated_scan_forward(cuda["z"], cuda["f"], bias, h0=h0, **kw)
    dirty_memory()
    _, df, dbias, _ = nsp.gated_scan_backward(cuda["dy"], dev(dh), cuda["z"], cuda["f"], bias, st, **kw)
    size = df.double().abs().sum((0, 1))
    bound = ((T / 8 + B + 16) * U + ROUND[dtype]) * size + 1e-30
    assert ((dbias.double() - df.double().sum((0, 1))).abs() <= bound).all()


def test_scan_with_a_bias_is_captured_in_a_graph(nsp):
    # the sums of the bias's gradient are a launch that may begin before the one it waits for ends
    z, dy = torch.randn(330, 70, 64).cuda(), torch.randn(330, 70, 64).cuda()
    bias = torch.rand(64).cuda()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(2):
            _, _, s = nsp.gated_scan_forward(z, z, bias)
            nsp.gated_scan_backward(dy, None, z, z, bias, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, states = nsp.gated_scan_forward(z, z, bias)
        back = nsp.gated_scan_backward(dy, None, z, z, bias, states)
    z.normal_(), dy.normal_(), bias.uniform_()
    graph.replay()
    torch.cuda.synchronize()
    want = nsp.gated_scan_forward(z, z, bias)
    for a, b in zip((y, h, states), want):
        assert torch.equal(a, b)
    for a, b in zip(back, nsp.gated_scan_backward(dy, None, z, z, bias, want[2])):
        assert torch.equal(a, b)


# ---- logits of 65 to 128 experts in 16 bits ----------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("E,k", [(65, 3), (100, 8), (127, 2), (128, 32)])
def test_route_16_bit_logits_of_a_thread_alone(nsp, E, k, dtype):
    """On both sides of as many tokens as fill the GPU with a thread each, to the bounds and
    with the bits of test_train_operators."""
    g = gen(E + k)
    x = torch.randn(21_011, E, generator=g).to(DTYPES[dtype])
    x[torch.rand(21_011, E, generator=g) < 0.1] = -INF
    x[7::113] = -INF
    x[9::113] = torch.finfo(DTYPES[dtype]).min
    doc = (torch.rand(21_011, generator=g) < 0.9).int() - 1
    check_route(nsp, x, k, doc, True, dtype)
    check_route(nsp, x[:19_456], k, None, False, dtype)
    xc, dw = x.cuda(), torch.randn(21_011, k, generator=g).cuda()
    many = nsp.route(xc, k)
    for n in (1, 77, 3000, 19_455):
        few = nsp.route(xc[:n], k)
        assert torch.equal(few.ids, many.ids[:n]) and torch.equal(few.weights, many.weights[:n])
        assert torch.equal(nsp.route_backward(xc[:n], few, dw[:n]),
                           nsp.route_backward(xc, many, dw)[:n])


# ---- the README's lines ---------------------------------------------------------------------------
def test_readme_lines_run_on_an_update(nsp):
    """On the arrays that the packer writes, and with the learned positions of the example."""
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    lines = text.split("### Training on the packed rows")[1].split("```python\n")[1].split("```")[0]
    from corpus import make_preset
    pk = nsp.Packer.from_corpus(make_preset("c1"))
    out = pk.step(0)
    v = {n: out[n][0] for n in ("pos", "doc", "mask")}
    B, T = v["pos"].shape
    v.update(z=torch.randn(B, T, 32).cuda(), f=torch.randn(B, T, 32).cuda(), bias=torch.zeros(32).cuda(),
             z1=torch.randn(B, 1, 32).cuda(), f1=torch.randn(B, 1, 32).cuda(),
             logits=torch.randn(B * T, 16).cuda(), student=torch.randn(B * T, 50).cuda(),
             w=torch.ones(B * T).cuda())
    v["top_logits"], v["top_ids"] = v["student"].topk(4, 1)
    exec(lines, v)
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        from packed_training_step import targets
    finally:
        sys.path.pop(0)
    _, learned = targets(out["tokens"][0], out["pos"][0], out["mask"][0])
    assert torch.equal(v["learned"], learned) and 0 < int(learned.sum()) < learned.numel()
    assert v["loss"].shape == (B * T,) and ((v["loss"] != 0) == (learned != 0)).all()
    pk.close()

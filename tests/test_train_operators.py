"""The training operators' kernels against plain 64-bit forms of their formulas.

Tolerances, with u = 2**-24 the rounding of a 32-bit float:

* scan: a state is a convex combination of inputs, so each step adds a few u of
  the largest input and forgets with the gates; over the lengths and gates here
  (memories up to some 400 steps) random roundings stay below 2e-5 of the
  result's norm.  A 16-bit output adds half a unit in its last place: up to
  2**-8 of each value in bfloat16, 2**-11 in float16.
* distillation: log q comes from products of up to about 40 in powers of two,
  so 40 * 2 u in an exponent, 5e-6, and as much again from the special function
  unit and the sums: 2e-5 of mq and of p, and 2e-5 absolute in a log.
* router: exponents up to about 30, as above: 1e-5 of each probability.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# the unit roundoff of the 16-bit types: 8 and 11 significant bits
ROUND = {"f32": 0.0, "bf16": 2.0**-8, "f16": 2.0**-11}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def nsp():
    import deterministic_packed_assembly_gb300 as m
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def dev(t):
    return None if t is None else t.cuda()


def close(got, want, rel, name, round_to=0.0, floor=0.0):
    """|got - want| within rel of the norm, and each value within its own
    rounding and `rel` of the largest; infinities and NaN in the same places."""
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), name
    if not fine.any():
        return
    d, w = (got - want)[fine], want[fine]
    top = float(w.abs().max()) + floor
    off = (d.abs() - round_to * w.abs() * 1.01).max()
    assert float(off) <= 20 * rel * top + 1e-30, (name, "one value", float(off), top)
    norm = float(w.norm())
    assert float(d.norm()) <= (rel + round_to) * norm + 20 * rel * floor + 1e-30, (
        name, "norm", float(d.norm()), norm)


# ---- gated linear recurrence ------------------------------------------------------
def scan_reference(z, f, bias, pos, doc, h0, dy=None, dh=None):
    z, f = z.double(), f.double()
    B, T, D = z.shape
    x = f if bias is None else f + bias.double()
    a, c = torch.sigmoid(x), torch.sigmoid(-x)
    start = torch.zeros(B, T, dtype=torch.bool) if pos is None else pos == 0
    skip = torch.zeros(B, T, dtype=torch.bool) if doc is None else doc < 0
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double().clone()
    y, before = torch.zeros(B, T, D, dtype=torch.float64), torch.zeros(B, T, D, dtype=torch.float64)
    for t in range(T):
        s, k = start[:, t, None], skip[:, t, None]
        p = torch.where(s, torch.zeros_like(h), h)
        new = a[:, t] * p + c[:, t] * z[:, t]
        h = torch.where(k, h, new)
        y[:, t] = torch.where(k, torch.zeros_like(new), new)
        before[:, t] = p
    out = dict(y=y, h_last=h)
    if dy is None:
        return out
    dy = dy.double()
    u = torch.zeros(B, D, dtype=torch.float64) if dh is None else dh.double().clone()
    dz, df = torch.zeros_like(y), torch.zeros_like(y)
    zero = torch.zeros_like(u)
    for t in range(T - 1, -1, -1):
        s, k = start[:, t, None], skip[:, t, None]
        d = dy[:, t] + u
        dz[:, t] = torch.where(k, zero, c[:, t] * d)
        df[:, t] = torch.where(k, zero, a[:, t] * c[:, t] * d * (before[:, t] - z[:, t]))
        u = torch.where(k, u, torch.where(s, zero, a[:, t] * d))
    out.update(dz=dz, df=df, dbias=df.sum((0, 1)), dh0=u)
    return out


def scan_inputs(B, T, D, dtype, seed, packed=True, state=True, joint=False, shift=0):
    """Inputs on the host, and z, f, dy on the GPU as the case lays them out."""
    g = gen(seed)
    dt = DTYPES[dtype]
    z, f, dy = (torch.randn(B, T, D, generator=g).to(dt) for _ in range(3))
    bias = torch.rand(D, generator=g) * 6
    h0 = torch.randn(B, D, generator=g) if state else None
    dh = torch.randn(B, D, generator=g) if state else None
    pos = doc = None
    if packed:
        start = torch.rand(B, T, generator=g) < 0.05
        t = torch.arange(T).expand(B, T)
        pos = (t + 5 - torch.where(start, t + 5, torch.zeros_like(t)).cummax(1).values).int()
        doc = start.int().cumsum(1).int()
        gone = torch.rand(B, T, generator=g) < 0.1
        doc = torch.where(gone, torch.full_like(doc, -1), doc)
        pos = torch.where(gone, torch.zeros_like(pos), pos)
    zc, fc, dyc = z.cuda(), f.cuda(), dy.cuda()
    if joint:
        both = torch.cat([zc, fc], 2)
        zc, fc = both[..., :D], both[..., D:]
    if shift:  # rows that do not start on a boundary of anything
        def moved(x):
            flat = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:]
            return flat.copy_(x.reshape(-1)).view(x.shape)
        zc, fc, dyc = moved(zc), moved(fc), moved(dyc)
    host = dict(z=z, f=f, bias=bias, pos=pos, doc=doc, h0=h0)
    return host, dict(z=zc, f=fc, dy=dyc), dy, dh


def check_scan(nsp, host, cuda, dy, dh, dtype):
    want = scan_reference(**host, dy=dy, dh=dh)
    kw = dict(pos=dev(host["pos"]), doc=dev(host["doc"]))
    h0, bias = dev(host["h0"]), dev(host["bias"])
    y, h, states = nsp.gated_scan_forward(cuda["z"], cuda["f"], bias, h0=h0, **kw)
    y2, h2 = nsp.gated_scan(cuda["z"], cuda["f"], bias, h0=h0, **kw)
    assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8))
    assert torch.equal(h.view(torch.uint8), h2.view(torch.uint8))
    close(y, want["y"], 2e-5, "y", ROUND[dtype])
    close(h, want["h_last"], 2e-5, "h_last")
    dz, df, dbias, dh0 = nsp.gated_scan_backward(cuda["dy"], dev(dh), cuda["z"], cuda["f"], bias,
                                                 states, **kw)
    floor = float(dy.double().abs().max()) if dy.numel() else 1.0
    close(dz, want["dz"], 2e-5, "dz", ROUND[dtype])
    close(df, want["df"], 2e-5, "df", ROUND[dtype])
    close(dbias, want["dbias"], 2e-5, "dbias", floor=floor)
    close(dh0, want["dh0"], 2e-5, "dh0", floor=floor)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,D", [
    (1, 1, 1), (3, 1, 64), (2, 2, 33), (2, 7, 2), (4, 8, 66), (3, 9, 130), (2, 63, 5), (2, 64, 64),
    (1, 65, 62), (2, 130, 31), (1, 517, 40), (5, 200, 96)])
def test_scan(nsp, B, T, D, dtype):
    check_scan(nsp, *scan_inputs(B, T, D, dtype, 7 * B + T + D), dtype)


@pytest.mark.parametrize("packed,state", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("T", [3, 150])
def test_scan_optional_inputs(nsp, T, packed, state):
    host, cuda, dy, dh = scan_inputs(2, T, 34, "f32", T, packed, state)
    check_scan(nsp, host, cuda, dy, dh, "f32")
    host["bias"] = None
    want = scan_reference(**host, dy=dy, dh=dh)
    kw = dict(pos=dev(host["pos"]), doc=dev(host["doc"]))
    y, h, states = nsp.gated_scan_forward(cuda["z"], cuda["f"], h0=dev(host["h0"]), **kw)
    close(y, want["y"], 2e-5, "y")
    got = nsp.gated_scan_backward(cuda["dy"], dev(dh), cuda["z"], cuda["f"], None, states, **kw)
    assert got[2] is None
    close(got[1], want["df"], 2e-5, "df")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("joint,shift", [(True, 0), (False, 1), (False, 2), (True, 1)])
def test_scan_strides_and_alignment(nsp, joint, shift, dtype):
    for T, D in ((5, 36), (150, 36), (150, 35)):
        check_scan(nsp, *scan_inputs(2, T, D, dtype, 11 + T + D, joint=joint, shift=shift), dtype)


def test_scan_time_major_and_sliced_inputs(nsp):
    # [T, B, D] tensors seen as [B, T, D], and every second channel block
    host, cuda, dy, dh = scan_inputs(3, 90, 32, "bf16", 5)
    for k in ("z", "f", "dy"):
        cuda[k] = cuda[k].transpose(0, 1).contiguous().transpose(0, 1)
    check_scan(nsp, host, cuda, dy, dh, "bf16")


@pytest.mark.parametrize("T", [600, 4000])
def test_scan_of_few_channels_is_split_along_time(nsp, T):
    # one row of 64 channels: a cluster of blocks shares the row
    check_scan(nsp, *scan_inputs(1, T, 64, "f32", T), "f32")
    check_scan(nsp, *scan_inputs(2, T + 37, 33, "bf16", T), "bf16")


@pytest.mark.parametrize("T", [6, 64, 129, 1000])
def test_scan_masks(nsp, T):
    """Rows of padding alone, padding first, one real position, sequences that
    start at every step, at no step, and exactly at the tiles' edges."""
    B, D = 7, 36
    host, cuda, dy, dh = scan_inputs(B, T, D, "f32", 100 + T)
    pos = torch.arange(1, T + 1).expand(B, T).clone().int()
    doc = torch.zeros(B, T, dtype=torch.int32)
    doc[0] = -1
    doc[1, : T // 2] = -1
    doc[2] = -1
    doc[2, T // 3] = 4
    pos[3] = 0
    pos[5, ::64] = 0
    pos[6, 7::8] = 0
    doc[6, 3::5] = -(2**31)
    host.update(pos=pos, doc=doc)
    check_scan(nsp, host, cuda, dy, dh, "f32")


@pytest.mark.parametrize("T", [8, 300])
def test_scan_ignores_what_padding_holds_and_keeps_documents_apart(nsp, T):
    host, cuda, dy, dh = scan_inputs(3, T, 34, "f32", 3 * T)
    host["pos"] = torch.arange(1, T + 1).expand(3, T).clone().int()
    host["pos"][:, T // 2] = 0
    host["doc"] = torch.zeros(3, T, dtype=torch.int32)
    host["doc"][:, 2] = -1
    host["doc"][0, T - 2:] = -1
    want = scan_reference(**host, dy=dy, dh=dh)
    gone = (host["doc"] < 0).cuda()
    for bad in (NAN, INF, -INF, torch.finfo(torch.float32).min):
        c = {k: torch.where(gone[..., None], torch.full_like(v, bad), v) for k, v in cuda.items()}
        kw = dict(pos=dev(host["pos"]), doc=dev(host["doc"]))
        y, h, st = nsp.gated_scan_forward(c["z"], c["f"], dev(host["bias"]), h0=dev(host["h0"]), **kw)
        got = nsp.gated_scan_backward(c["dy"], dev(dh), c["z"], c["f"], dev(host["bias"]), st, **kw)
        for g, name in zip((y, h, *got), ("y", "h_last", "dz", "df", "dbias", "dh0")):
            close(g, want[name], 2e-5, name)
    # a NaN in the first document reaches no position of the second one
    z = cuda["z"].clone()
    z[1, 0] = NAN
    y, h, st = nsp.gated_scan_forward(z, cuda["f"], dev(host["bias"]), h0=dev(host["h0"]),
                                      pos=dev(host["pos"]), doc=dev(host["doc"]))
    assert torch.isnan(y[1, : T // 2][host["doc"][1, : T // 2] >= 0]).all()
    close(y[:, T // 2:], want["y"][:, T // 2:], 2e-5, "y after")
    close(h, want["h_last"], 2e-5, "h_last after")
    dy2 = cuda["dy"].clone()
    dy2[1, T - 1] = NAN
    got = nsp.gated_scan_backward(dy2, dev(dh), cuda["z"], cuda["f"], dev(host["bias"]), nsp.
                                  gated_scan_forward(cuda["z"], cuda["f"], dev(host["bias"]),
                                                     h0=dev(host["h0"]), pos=dev(host["pos"]),
                                                     doc=dev(host["doc"]))[2],
                                  pos=dev(host["pos"]), doc=dev(host["doc"]))
    close(got[0][:, : T // 2], want["dz"][:, : T // 2], 2e-5, "dz before")
    assert torch.isnan(got[0][1, T // 2:][host["doc"][1, T // 2:] >= 0]).all()


def test_scan_extreme_gates(nsp):
    # gates at 0 and 1 exactly, and beyond what exp holds
    f = torch.tensor([0.0, 30.0, -30.0, 90.0, -90.0, 200.0, -200.0, INF, -INF])
    f = f[None, :, None].expand(2, 9, 6).contiguous()
    host = dict(z=torch.randn(2, 9, 6, generator=gen(1)), f=f, bias=torch.zeros(6), pos=None,
                doc=None, h0=torch.randn(2, 6, generator=gen(2)))
    cuda = dict(z=host["z"].cuda(), f=f.cuda(), dy=torch.ones(2, 9, 6).cuda())
    check_scan(nsp, host, cuda, torch.ones(2, 9, 6), torch.randn(2, 6, generator=gen(3)), "f32")


def test_scan_empty(nsp):
    h0 = torch.randn(2, 5).cuda()
    z = torch.empty(2, 0, 5, device="cuda")
    y, h, states = nsp.gated_scan_forward(z, z, h0=h0, bias=torch.zeros(5).cuda())
    assert y.shape == (2, 0, 5) and torch.equal(h, h0)
    dz, df, dbias, dh0 = nsp.gated_scan_backward(z, h0, z, z, torch.zeros(5).cuda(), states)
    assert torch.equal(dh0, h0) and torch.equal(dbias, torch.zeros(5).cuda())
    z = torch.empty(0, 70, 5, device="cuda")
    y, h, states = nsp.gated_scan_forward(z, z, torch.zeros(5).cuda())
    assert h.shape == (0, 5)
    assert torch.equal(nsp.gated_scan_backward(z, None, z, z, torch.zeros(5).cuda(), states)[2],
                       torch.zeros(5).cuda())


def test_scan_token_by_token_equals_the_whole_row(nsp):
    # the serving form: T = 1, the state handed on (in place through the C ABI)
    host, cuda, _, _ = scan_inputs(3, 70, 34, "f32", 9)
    kw = dict(bias=dev(host["bias"]))
    y, h_last = nsp.gated_scan(cuda["z"], cuda["f"], pos=dev(host["pos"]), doc=dev(host["doc"]),
                               h0=dev(host["h0"]), **kw)
    h = dev(host["h0"])
    for t in range(70):
        yt, h = nsp.gated_scan(cuda["z"][:, t:t + 1], cuda["f"][:, t:t + 1], h0=h,
                               pos=host["pos"][:, t:t + 1].contiguous().cuda(),
                               doc=host["doc"][:, t:t + 1].contiguous().cuda(), **kw)
        close(yt[:, 0], y[:, t].double().cpu(), 2e-5, f"y {t}")
    close(h, h_last.double().cpu(), 2e-5, "h_last")
    for T in (4, 70):  # h_last written over h0
        h = dev(host["h0"]).clone()
        want = nsp.gated_scan(cuda["z"][:, :T], cuda["f"][:, :T], h0=h, **kw)
        out = torch.empty_like(want[0])
        zt, ft = cuda["z"][:, :T], cuda["f"][:, :T]
        inputs = nsp._lib.ns_scan_inputs(zt.data_ptr(), ft.data_ptr(), zt.stride(0), zt.stride(1),
                                         ft.stride(0), ft.stride(1), kw["bias"].data_ptr(), None,
                                         None, 3, T, 34, nsp.NS_F32)
        nsp.ns_scan_forward(inputs, h.data_ptr(), out.data_ptr(), h.data_ptr(), None,
                            torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("T", [1, 7, 8, 9, 24, 31, 32, 33, 70, 700])
def test_scan_rows_do_not_depend_on_the_other_rows(nsp, T):
    # few rows and many take other kernels and other clusters: the same bits
    host, cuda, dy, dh = scan_inputs(60, T, 1300, "bf16", T)
    kw = dict(pos=dev(host["pos"]), doc=dev(host["doc"]))
    bias, h0, dhc = dev(host["bias"]), dev(host["h0"]), dev(dh)
    y, h, st = nsp.gated_scan_forward(cuda["z"], cuda["f"], bias, h0=h0, **kw)
    back = nsp.gated_scan_backward(cuda["dy"], dhc, cuda["z"], cuda["f"], bias, st, **kw)
    for rows in (slice(3, 4), slice(17, 22)):
        kw = dict(pos=dev(host["pos"])[rows], doc=dev(host["doc"])[rows])
        part = dict(z=cuda["z"][rows], f=cuda["f"][rows])
        y1, h1, s1 = nsp.gated_scan_forward(part["z"], part["f"], bias, h0=h0[rows], **kw)
        one = nsp.gated_scan_backward(cuda["dy"][rows], dhc[rows], part["z"], part["f"], bias, s1, **kw)
        assert torch.equal(y1, y[rows]) and torch.equal(h1, h[rows]) and torch.equal(s1, st[rows])
        for a, b, name in zip(one, back, ("dz", "df", "dbias", "dh0")):
            assert name == "dbias" or torch.equal(a, b[rows]), name


def test_route_tokens_do_not_depend_on_the_other_tokens(nsp):
    for E, k in ((64, 8), (100, 4), (250, 3), (1000, 8)):
        x = torch.randn(30_000, E, generator=gen(E)).cuda()
        dw = torch.randn(30_000, k, generator=gen(k)).cuda()
        many = nsp.route(x, k)
        for n in (1, 77, 2000):
            few = nsp.route(x[:n], k)
            assert torch.equal(few.ids, many.ids[:n]) and torch.equal(few.weights, many.weights[:n])
            assert torch.equal(nsp.route_backward(x[:n], few, dw[:n]),
                               nsp.route_backward(x, many, dw)[:n])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_route_16_bit_tokens_do_not_depend_on_the_other_tokens(nsp, dtype):
    for E, k in ((61, 2), (250, 3), (1000, 8)):
        x = torch.randn(30_000, E, generator=gen(E)).to(DTYPES[dtype]).cuda()
        dw = torch.randn(30_000, k, generator=gen(k)).cuda()
        many = nsp.route(x, k)
        for n in (1, 77, 2000):
            few = nsp.route(x[:n], k)
            assert torch.equal(few.ids, many.ids[:n]) and torch.equal(few.weights, many.weights[:n])
            assert torch.equal(nsp.route_backward(x[:n], few, dw[:n]),
                               nsp.route_backward(x, many, dw)[:n])


def test_scan_offsets_past_32_bits(nsp):
    B, T, D = 3, 360_001, 2048  # 2.2e9 elements
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    z = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    f = torch.empty_like(z).normal_(generator=g)
    y, h, states = nsp.gated_scan_forward(z, f)
    y1, h1, s1 = nsp.gated_scan_forward(z[2:], f[2:])
    assert torch.equal(y[2:], y1) and torch.equal(h[2:], h1)
    # the sums of dbias are split otherwise for one row, the others are not
    dz, df, _, dh0 = nsp.gated_scan_backward(y, h, z, f, None, states)
    dz1, df1, _, dh1 = nsp.gated_scan_backward(y1, h1, z[2:], f[2:], None, s1)
    assert torch.equal(dz[2:], dz1) and torch.equal(df[2:], df1) and torch.equal(dh0[2:], dh1)


def directional(f, x, v, eps):
    return (f(x + eps * v) - f(x - eps * v)) / (2 * eps)


def test_scan_gradients_against_differences(nsp):
    """Central differences of the kernel's own forward pass along the gradient:
    a step of 0.02 truncates about 1e-4 of it and the 32-bit sums' rounding over
    the step is below 1e-4: 5e-3 is asked for."""
    host, cuda, dy, dh = scan_inputs(2, 90, 34, "f32", 21)
    pos, doc = dev(host["pos"]), dev(host["doc"])
    leaves = [cuda["z"].clone(), cuda["f"].clone(), dev(host["bias"]), dev(host["h0"])]
    for t in leaves:
        t.requires_grad_()

    def value(ts):
        y, h = nsp.gated_scan(ts[0], ts[1], ts[2], pos=pos, doc=doc, h0=ts[3])
        return (y.double() * cuda["dy"].double()).sum() + (h.double() * dh.cuda().double()).sum()

    grads = torch.autograd.grad(value(leaves), leaves)
    explicit = nsp.gated_scan_backward(
        cuda["dy"], dev(dh), leaves[0], leaves[1], leaves[2],
        nsp.gated_scan_forward(*leaves[:3], pos=pos, doc=doc, h0=leaves[3])[2], pos=pos, doc=doc)
    for g, e in zip(grads, explicit):
        close(g, e.double().cpu(), 1e-6, "autograd")
    plain = [t.detach() for t in leaves]
    for i, g in enumerate(grads):
        v = g / g.abs().max()

        def at(x, i=i):
            return float(value([x if j == i else t for j, t in enumerate(plain)]))

        slope = float((g.double() * v.double()).sum())
        assert abs(directional(at, plain[i], v, 0.02) - slope) <= 5e-3 * abs(slope), i


def test_scan_autograd_of_one_output(nsp):
    host, cuda, _, _ = scan_inputs(2, 20, 6, "f32", 2)
    z = cuda["z"].clone().requires_grad_()
    y, h = nsp.gated_scan(z, cuda["f"])
    (g1,) = torch.autograd.grad(h.sum(), z, retain_graph=True)  # no gradient of y
    (g2,) = torch.autograd.grad(y.sum(), z)                     # an expanded one of y
    one = dict(host, bias=None, pos=None, doc=None, h0=None)
    ones = torch.ones(2, 6)
    zero = torch.zeros(2, 20, 6)
    close(g1, scan_reference(**one, dy=zero, dh=ones)["dz"], 2e-5, "h")
    close(g2, scan_reference(**one, dy=zero + 1, dh=None)["dz"], 2e-5, "y")


# ---- distillation -------------------------------------------------------------------
def distill_reference(logits, top, ids, mask, temp, lse, weight):
    x = logits.double() / temp
    N, V = x.shape
    ids = ids.long()
    ok = (ids >= 0) & (ids < V)
    t = torch.where(ok, top.double() / temp, torch.full(top.shape, -INF, dtype=torch.float64))
    p = (torch.softmax(t, 1) if lse is None else torch.exp(t - lse.double()[:, None]))
    p = torch.where(ok, p, torch.zeros_like(p))
    p = torch.where((t == -INF).all(1, keepdim=True), torch.zeros_like(p), p)
    full = torch.zeros(N, V, dtype=torch.float64).scatter_add_(1, ids.clamp(0, V - 1), p)
    top_x = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top_x == -INF, torch.zeros_like(top_x), top_x))
    s = e.sum(1, keepdim=True)
    q = torch.where(s == 0, torch.zeros_like(e), e / s)
    log_q = torch.where(x == -INF, x, x - top_x - torch.log(s))
    log_p = t - torch.logsumexp(t, 1, keepdim=True) if lse is None else t - lse.double()[:, None]
    terms = p * (log_p - log_q.gather(1, ids.clamp(0, V - 1)))
    loss = temp**2 * torch.where(p == 0, torch.zeros_like(terms), terms).sum(1)
    m = p.sum(1, keepdim=True)
    g = temp * (torch.where(m == 0, torch.zeros_like(q), m * q) - full)
    if weight is not None:
        g = g * weight.double()[:, None]
    if mask is not None:
        loss = torch.where(mask != 0, loss, torch.zeros_like(loss))
        g = torch.where((mask != 0)[:, None], g, torch.zeros_like(g))
    return loss, g


def distill_inputs(N, V, K, dtype, seed, tail=False, tdtype="f32", learned=1.0, temp=1.0):
    g = gen(seed)
    logits = (torch.randn(N, V, generator=g) * 2.5).to(DTYPES[dtype])
    noisy = logits.float() + torch.randn(N, V, generator=g)
    top, ids = noisy.topk(K, 1)
    top = top.to(DTYPES[tdtype])
    lse = None
    if tail:
        lse = torch.logsumexp(top.float() / temp, 1) + 0.3 * torch.rand(N, generator=g)
    mask = None
    if learned < 1:
        mask = (torch.rand(N, generator=g) < learned).to(torch.uint8)
    weight = torch.randn(N, generator=g)
    return dict(logits=logits, top=top, ids=ids.int(), mask=mask, temp=temp, lse=lse, weight=weight)


def run_distill(nsp, c, logits=None, out=None):
    logits = dev(c["logits"]) if logits is None else logits
    kw = dict(mask=dev(c["mask"]), temperature=c["temp"], teacher_lse=dev(c["lse"]))
    loss = nsp.distill_loss(logits, dev(c["top"]), dev(c["ids"]), **kw)
    both = nsp.distill_grad(logits, dev(c["top"]), dev(c["ids"]), weight=dev(c["weight"]), out=out,
                            **kw)
    assert torch.equal(loss.view(torch.int32), both[0].view(torch.int32))
    return both


def check_distill(nsp, c, dtype, logits=None, out=None):
    want_loss, want_g = distill_reference(**c)
    loss, g = run_distill(nsp, c, logits, out)
    t2 = c["temp"] ** 2
    got, want = loss.double().cpu(), want_loss
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert (got - want)[fine].abs().max().item() <= 2e-5 * t2 * (1 + want[fine].abs().max().item())
    scale = c["temp"] * (1.0 if c["weight"] is None else c["weight"].double().abs()[:, None])
    bound = 2e-5 * (want_g.abs() + 2 * torch.where(want_g < 0, scale * torch.ones_like(want_g),
                                                   torch.zeros_like(want_g)))
    bound += 2e-5 * scale * 1e-3 + ROUND[dtype] * 1.01 * want_g.abs()
    if dtype == "f16":
        bound += 2.0**-24  # a unit of its subnormal numbers
    assert not torch.isnan(g).any()
    assert ((g.double().cpu() - want_g).abs() <= bound).all()
    return loss, g


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 8, 8), (3, 100, 5),
                                   (2, 1003, 33), (2, 4099, 300), (2, 50257, 64), (1, 32768, 1024)])
def test_distill(nsp, N, V, K, dtype):
    check_distill(nsp, distill_inputs(N, V, K, dtype, N + V + K), dtype)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temp", [0.5, 1.0, 3.0])
@pytest.mark.parametrize("tdtype", ["f32", "bf16", "f16"])
def test_distill_temperature_tail_and_mask(nsp, tail, temp, tdtype):
    c = distill_inputs(9, 517, 12, "bf16", 3, tail, tdtype, 0.6, temp)
    c["mask"][0], c["mask"][1] = 1, 0
    check_distill(nsp, c, "bf16")
    c["weight"] = None
    check_distill(nsp, c, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40_000, 70_001, 150_000, 260_001, 400_000])
def test_distill_rows_in_several_blocks(nsp, V, dtype):
    # every cluster size; the widest rows fill a block's shared memory alone
    check_distill(nsp, distill_inputs(2, V, 40, dtype, V), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift,row,out_row,out_shift", [
    (0, 1003, 1003, 0), (1, 1005, 1003, 0), (3, 1001, 1001, 3), (0, 1008, 1008, 1),
    (8, 1001, 1016, 0)])
def test_distill_strides_and_alignment(nsp, shift, row, out_row, out_shift, dtype):
    N, V = 6, 1001
    c = distill_inputs(N, V, 9, dtype, shift + row, learned=0.7)
    c["mask"][0] = 1
    flat = torch.full((N * row + shift,), NAN, dtype=DTYPES[dtype], device="cuda")
    logits = flat[shift:].view(N, row)[:, :V]
    logits.copy_(c["logits"])
    # columns beyond V, and what lies around the gradient, are left alone
    flat_out = torch.full((N * out_row + out_shift + 8,), 77.0, dtype=DTYPES[dtype], device="cuda")
    out = flat_out[out_shift:out_shift + N * out_row].view(N, out_row)[:, :V]
    _, g = check_distill(nsp, c, dtype, logits, out)
    assert g.data_ptr() == out.data_ptr()
    out.fill_(77.0)
    assert (flat_out == 77.0).all()


@pytest.mark.parametrize("V", [1001, 64_000, 128_256])
def test_distill_gradient_in_the_logits_place(nsp, V):
    c = distill_inputs(3, V, 20, "bf16", 1, learned=0.9)
    c["mask"][0], c["mask"][1] = 1, 0
    loss, g = run_distill(nsp, c)
    logits = dev(c["logits"])
    both = nsp.distill_grad(logits, dev(c["top"]), dev(c["ids"]), mask=dev(c["mask"]),
                            weight=dev(c["weight"]), out=logits)
    assert both[1].data_ptr() == logits.data_ptr()
    assert torch.equal(both[0], loss) and torch.equal(logits, g)


def test_distill_repeated_and_absent_ids(nsp):
    c = distill_inputs(6, 300, 24, "f32", 8)
    c["ids"][0, :] = 17                      # one id for all entries
    c["ids"][1, 3:9] = c["ids"][1, 2]        # some repeated
    c["ids"][2, ::2] = -1                    # absent
    c["ids"][3, 5] = 300
    c["ids"][3, 6] = 2**31 - 1
    c["ids"][4, :] = -5                      # none left: nothing to learn
    check_distill(nsp, c, "f32")
    loss, g = run_distill(nsp, c)
    assert loss[4] == 0 and (g[4] == 0).all()
    wide = dict(c, ids=c["ids"].long())
    wide["ids"][5, 0] = 2**40 + 3            # absent, not 3
    c["ids"][5, 0] = -1
    a, b = run_distill(nsp, c), run_distill(nsp, wide)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("V", [300, 90_000])
def test_distill_infinities(nsp, V):
    c = distill_inputs(6, V, 12, "f32", 4)
    c["logits"][0, 5:200] = -INF             # masked vocabulary, some of it the teacher's
    c["ids"][0, 0] = 7
    keep = torch.ones(V, dtype=torch.bool)
    keep[c["ids"][1].long()] = False
    c["logits"][1, keep] = -INF              # nothing but the teacher's entries
    c["top"][2, 3:] = -INF                   # entries of probability 0 ...
    c["logits"][2, c["ids"][2, 5].long()] = -INF  # ... add nothing where q is 0
    c["top"][3] = -INF                       # a teacher without any entry
    c["logits"][4] = -INF                    # a student without any
    c["logits"][5] = torch.finfo(torch.float32).min
    loss, g = check_distill(nsp, c, "f32")
    assert math.isinf(loss[0]) and loss[3] == 0 and (g[3] == 0).all() and math.isinf(loss[4])


def test_distill_does_not_read_unlearned_rows(nsp):
    c = distill_inputs(8, 2000, 10, "bf16", 6, learned=0.5)
    c["mask"][0], c["mask"][1] = 0, 1
    want = run_distill(nsp, c)
    off = c["mask"] == 0
    for bad in (NAN, INF, -INF):
        d = dict(c, logits=c["logits"].clone(), top=c["top"].clone(), weight=c["weight"].clone())
        d["logits"][off], d["top"][off], d["weight"][off] = bad, bad, bad
        d["lse"] = None
        got = run_distill(nsp, d)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    as_bool = dict(c, mask=c["mask"] != 0)
    got = run_distill(nsp, as_bool)
    assert torch.equal(got[1], want[1])


def test_distill_nan_stays_in_its_row(nsp):
    c = distill_inputs(4, 700, 10, "f32", 12)
    want = run_distill(nsp, c)
    c["logits"][2, 333] = NAN
    loss, g = run_distill(nsp, c)
    assert torch.isnan(loss[2]) and torch.isnan(g[2]).all()
    for r in (0, 1, 3):
        assert torch.equal(loss[r], want[0][r]) and torch.equal(g[r], want[1][r])


def test_distill_empty_batch(nsp):
    z = torch.empty(0, 10, device="cuda")
    loss, g = nsp.distill_grad(z, z[:, :3], torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert loss.shape == (0,) and g.shape == (0, 10)


def test_distill_offsets_past_32_bits(nsp):
    N, V, K = 17_000, 128_256, 8  # 2.18e9 elements
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    logits = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, V, (N, K), generator=g, device="cuda")
    top = torch.empty(N, K, device="cuda").normal_(generator=g)
    loss, d = nsp.distill_grad(logits, top, ids)
    l2, d2 = nsp.distill_grad(logits[-300:], top[-300:], ids[-300:])
    assert torch.equal(loss[-300:], l2) and torch.equal(d[-300:], d2)


def test_distill_gradient_against_differences(nsp):
    """As for the scan: a step of 0.02 along the gradient, 5e-3."""
    for temp, tail in ((1.0, False), (2.0, True)):
        c = distill_inputs(6, 150, 12, "f32", 31, tail, learned=0.8, temp=temp)
        c["mask"][0] = 1
        kw = dict(mask=dev(c["mask"]), temperature=temp, teacher_lse=dev(c["lse"]))
        top, ids, w = dev(c["top"]), dev(c["ids"]), dev(c["weight"])
        x = dev(c["logits"]).requires_grad_()

        def value(x):
            return (nsp.distill_loss(x, top, ids, **kw).double() * w.double()).sum()

        (g,) = torch.autograd.grad(value(x), x)
        _, e = nsp.distill_grad(x.detach(), top, ids, weight=w, **kw)
        assert torch.equal(g, e)
        v = g / g.abs().max()
        slope = float((g.double() * v.double()).sum())
        got = directional(lambda y: float(value(y)), x.detach(), v, 0.02)
        assert abs(got - slope) <= 5e-3 * abs(slope)


# ---- router ---------------------------------------------------------------------------
def route_reference(logits, k, doc, normalize, dw=None, dl=None):
    x = logits.double()
    N, E = x.shape
    real = torch.ones(N, dtype=torch.bool) if doc is None else doc >= 0
    top = x.amax(1, keepdim=True)
    real = real & (top[:, 0] > -INF)
    x = torch.where(real[:, None], x, torch.zeros_like(x))
    p = torch.softmax(x, 1)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    ok = (x.gather(1, order) > -INF) & real[:, None]
    ids = torch.where(ok, order, torch.full_like(order, -1))
    at = torch.where(ok, p.gather(1, order), torch.zeros(N, k, dtype=torch.float64))
    total = at.sum(1, keepdim=True)
    w = torch.where(ok, at / total, at) if normalize else at
    counts = torch.bincount(ids[ok], minlength=E)
    M = int(real.sum())
    mass = p[real].sum(0)
    coef = E / (k * M * M) if M else 0.0
    loss = coef * (counts.double() * mass).sum()
    out = dict(ids=ids.int(), weights=w, counts=counts.int(), tokens=M, loss=loss)
    if dw is None and dl is None:
        return out
    g = torch.zeros(N, E, dtype=torch.float64)
    if dl is not None:
        g += float(dl) * coef * counts.double()
    if dw is not None:
        dw = torch.where(ok, dw.double(), torch.zeros(N, k, dtype=torch.float64))
        if normalize:
            dw = torch.where(ok, (dw - (w * dw).sum(1, keepdim=True)) / total, dw)
        g = g.scatter_add(1, order, dw)
    d = p * (g - (p * g).sum(1, keepdim=True))
    out["dlogits"] = torch.where(real[:, None], d, torch.zeros_like(d))
    # what the terms of a gradient add up to, without their signs
    size = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    out["size"] = torch.where(real[:, None], size, torch.zeros_like(size))
    return out


def check_route(nsp, logits, k, doc, normalize, dtype, cuda=None, seed=0):
    N, E = logits.shape
    g = gen(seed)
    dw, dl = torch.randn(N, k, generator=g), torch.tensor(0.7)
    want = route_reference(logits, k, doc, normalize, dw, dl)
    cuda = logits.cuda() if cuda is None else cuda
    r = nsp.route(cuda, k, doc=dev(doc), normalize=normalize)
    assert torch.equal(r.ids.cpu(), want["ids"])
    assert torch.equal(r.counts.cpu(), want["counts"]) and int(r.tokens) == want["tokens"]
    assert ((r.weights.double().cpu() - want["weights"]).abs() <= 1e-5 * want["weights"]).all()
    assert abs(float(r.loss) - float(want["loss"])) <= 1e-5 * abs(float(want["loss"]))
    d = nsp.route_backward(cuda, r, dw.cuda(), dl.cuda(), doc=dev(doc), normalize=normalize)
    assert d.dtype == cuda.dtype

    def near(got, w):
        bound = 2e-5 * w["size"] + ROUND[dtype] * 1.01 * w["dlogits"].abs()
        bound += 2.0**-24 if dtype == "f16" else 1e-37
        assert ((got.double().cpu() - w["dlogits"]).abs() <= bound).all()

    near(d, want)
    near(nsp.route_backward(cuda, r, None, dl.cuda(), doc=dev(doc), normalize=normalize),
         route_reference(logits, k, doc, normalize, None, dl))
    near(nsp.route_backward(cuda, r, dw.cuda(), None, doc=dev(doc), normalize=normalize),
         route_reference(logits, k, doc, normalize, dw, None))
    return r


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,E,k", [
    (1, 1, 1), (5, 2, 1), (7, 3, 3), (33, 8, 2), (70, 16, 4), (65, 17, 17), (130, 32, 6),
    (64, 64, 8), (301, 60, 6), (90, 100, 8), (140, 128, 32), (77, 129, 1), (257, 256, 8),
    (50, 300, 5), (41, 512, 10), (30, 1000, 32), (29, 1024, 7)])
def test_route(nsp, N, E, k, dtype):
    g = gen(N + E + k)
    logits = (torch.randn(N, E, generator=g) * 2).to(DTYPES[dtype])
    doc = (torch.rand(N, generator=g) < 0.8).int() - 1
    check_route(nsp, logits, k, doc, True, dtype)
    check_route(nsp, logits, k, None, False, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,E", [(20_011, 64), (5_003, 200), (3_001, 1024), (100_003, 8)])
def test_route_many_tokens(nsp, N, E, dtype):
    g = gen(E)
    logits = (torch.randn(N, E, generator=g) + torch.randn(1, E, generator=g)).to(DTYPES[dtype])
    doc = (torch.rand(N, generator=g) < 0.9).int() - 1
    check_route(nsp, logits, min(E, 4), doc, True, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,E,k", [(11_003, 251, 8), (11_003, 250, 2), (10_001, 256, 8), (5_001, 514, 3)])
def test_route_many_tokens_of_many_experts(nsp, N, E, k, dtype):
    # masked experts, rows without any, rows of the lowest value, padding that holds anything
    g = gen(E + k)
    logits = torch.randn(N, E, generator=g).to(DTYPES[dtype])
    logits[torch.rand(N, E, generator=g) < 0.2] = -INF
    logits[::97] = -INF
    logits[5::97] = torch.finfo(DTYPES[dtype]).min
    doc = (torch.rand(N, generator=g) < 0.9).int() - 1
    check_route(nsp, logits, k, doc, True, dtype)
    bad = logits.clone()
    bad[doc < 0] = NAN
    a, b = nsp.route(logits.cuda(), k, doc=doc.cuda()), nsp.route(bad.cuda(), k, doc=doc.cuda())
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,k", [(8, 4), (64, 8), (250, 16), (600, 8)])
def test_route_ties_go_to_the_lowest_index(nsp, E, k, dtype):
    g = gen(E + k)
    logits = torch.randint(-2, 3, (200, E), generator=g).to(DTYPES[dtype])
    logits[torch.rand(200, E, generator=g) < 0.3] *= -1.0  # zeros of both signs among them
    logits[0] = 0
    logits[1] = torch.finfo(DTYPES[dtype]).min
    check_route(nsp, logits, k, None, True, dtype)


@pytest.mark.parametrize("E,k", [(6, 4), (64, 8), (300, 3)])
def test_route_masked_experts_and_rows(nsp, E, k):
    g = gen(E)
    logits = torch.randn(40, E, generator=g)
    logits[torch.rand(40, E, generator=g) < 0.5] = -INF
    logits[3] = -INF                      # no expert at all
    logits[4] = -INF
    logits[4, E - 1] = 0.5                # one expert
    logits[5] = torch.finfo(torch.float32).min
    logits[6] = 1e30                      # large, all equal
    doc = torch.zeros(40, dtype=torch.int32)
    doc[7] = -1
    for normalize in (True, False):
        check_route(nsp, logits, k, doc, normalize, "f32")
    bad = logits.clone()
    for v in (NAN, INF, 3.0):             # padding holds anything
        bad[7] = v
        a = nsp.route(logits.cuda(), k, doc=doc.cuda())
        b = nsp.route(bad.cuda(), k, doc=doc.cuda())
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        dw = torch.randn(40, k, generator=gen(1))
        da = nsp.route_backward(logits.cuda(), a, dw.cuda(), None, doc=doc.cuda())
        dw[7], dw[3] = v, v               # and so do gradients of weights that are not there
        dw[4, 1:] = v
        db = nsp.route_backward(bad.cuda(), b, dw.cuda(), None, doc=doc.cuda())
        assert torch.equal(da, db)


def test_route_all_padding_and_empty(nsp):
    x = torch.randn(9, 12).cuda()
    doc = torch.full((9,), -1, dtype=torch.int32).cuda()
    r = nsp.route(x, 3, doc=doc)
    assert int(r.tokens) == 0 and float(r.loss) == 0 and (r.ids == -1).all()
    assert (r.weights == 0).all() and (r.counts == 0).all()
    d = nsp.route_backward(x, r, torch.ones(9, 3).cuda(), torch.ones(()).cuda(), doc=doc)
    assert (d == 0).all()
    r = nsp.route(x[:0], 3)
    assert r.ids.shape == (0, 3) and int(r.tokens) == 0 and float(r.loss) == 0
    assert (r.counts == 0).all()
    assert nsp.route_backward(x[:0], r, None, torch.ones(()).cuda()).shape == (0, 12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift,row", [(0, 72), (1, 65), (4, 68), (3, 64)])
def test_route_strides_and_alignment(nsp, shift, row, dtype):
    x = torch.randn(50, 64, generator=gen(row)).to(DTYPES[dtype])
    flat = torch.full((50 * row + shift,), NAN, dtype=DTYPES[dtype], device="cuda")
    cuda = flat[shift:].view(50, row)[:, :64]
    cuda.copy_(x)
    check_route(nsp, x, 8, None, True, dtype, cuda)


def test_route_balance_is_one_when_even(nsp):
    E, k = 16, 2
    logits = torch.zeros(E, E)
    for n in range(E):  # token n prefers experts n and n + 1
        logits[n, n] = logits[n, (n + 1) % E] = 20.0
    r = nsp.route(logits.cuda(), k)
    assert (r.counts == k).all() and abs(float(r.loss) - 1.0) < 1e-6


def test_route_nan_stays_in_its_row(nsp):
    x = torch.randn(40, 64, generator=gen(3))
    want = nsp.route(x.cuda(), 8)
    x[11, 5] = NAN
    r = nsp.route(x.cuda(), 8)
    keep = torch.arange(40) != 11
    assert torch.equal(r.ids.cpu()[keep], want.ids.cpu()[keep])
    assert torch.equal(r.weights.cpu()[keep], want.weights.cpu()[keep])
    assert torch.isnan(r.loss) and ((r.ids[11] >= 0) & (r.ids[11] < 64)).all()
    assert torch.isnan(r.weights[11]).all()


@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradients_against_differences(nsp, normalize):
    """Along the gradient, with a step so small that no choice of experts changes
    and central differences of O(1) functions in 32 bits hold 5e-3."""
    g = gen(77)
    x = (torch.randperm(40 * 24, generator=g).float().view(40, 24) / 120.0).cuda().requires_grad_()
    doc = ((torch.rand(40, generator=g) < 0.8).int() - 1).cuda()
    dw = torch.randn(40, 4, generator=g).cuda()

    def value(x):
        r = nsp.route(x, 4, doc=doc, normalize=normalize)
        return (r.weights.double() * dw.double()).sum() + 30.0 * r.loss.double()

    (grad,) = torch.autograd.grad(value(x), x)
    r = nsp.route(x.detach(), 4, doc=doc, normalize=normalize)
    e = nsp.route_backward(x.detach(), r, dw, torch.tensor(30.0).cuda(), doc=doc,
                           normalize=normalize)
    close(grad, e.double().cpu(), 1e-6, "autograd")
    v = grad / grad.abs().max()
    slope = float((grad.double() * v.double()).sum())
    got = directional(lambda y: float(value(y)), x.detach(), v, 4e-3)  # logits are 1/120 apart
    assert abs(got - slope) <= 5e-3 * abs(slope)


# ---- all of them -------------------------------------------------------------------------
def test_same_bits_every_time_and_on_every_stream(nsp):
    host, cuda, dy, dh = scan_inputs(1, 3000, 130, "bf16", 1)
    kw = dict(pos=dev(host["pos"]), doc=dev(host["doc"]))
    c = distill_inputs(300, 5000, 30, "bf16", 2)
    c["ids"][0, 4:20] = c["ids"][0, 0]
    cc = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    x = torch.randn(30_000, 64, generator=gen(3)).cuda()
    dw, dl = torch.randn(30_000, 8, generator=gen(4)).cuda(), torch.ones(()).cuda()
    bias, dhc = dev(host["bias"]), dev(dh)

    def once():
        y, h, st = nsp.gated_scan_forward(cuda["z"], cuda["f"], bias, **kw)
        out = [y, h, st, *nsp.gated_scan_backward(cuda["dy"], dhc, cuda["z"], cuda["f"], bias, st,
                                                  **kw)]
        out += nsp.distill_grad(cc["logits"], cc["top"], cc["ids"], weight=cc["weight"])
        r = nsp.route(x, 8)
        return out + [*r, nsp.route_backward(x, r, dw, dl)]

    first = once()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    again = []
    for s in streams:
        with torch.cuda.stream(s):
            again.append(once())
    torch.cuda.synchronize()
    for other in again:
        for a, b in zip(first, other):
            assert torch.equal(a.view(torch.uint8) if a.dim() else a, b.view(torch.uint8) if b.dim() else b)


def test_calls_are_captured_in_a_graph(nsp):
    # nothing in a call waits, copies to the host or allocates behind PyTorch's back
    z = torch.randn(2, 200, 64).cuda()
    x = torch.randn(3000, 64).cuda()
    top, ids = x.topk(4, 1)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(2):
            nsp.gated_scan_forward(z, z)
            nsp.route(x, 4)
            nsp.distill_grad(x, top, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, states = nsp.gated_scan_forward(z, z)
        back = nsp.gated_scan_backward(y, h, z, z, None, states)
        r = nsp.route(x, 4)
        loss, d = nsp.distill_grad(x, top, ids)
    z.normal_()
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    want = nsp.gated_scan_forward(z, z)
    assert torch.equal(y, want[0])
    assert torch.equal(back[0], nsp.gated_scan_backward(y, h, z, z, None, states)[0])
    r2 = nsp.route(x, 4)
    assert torch.equal(r.ids, r2.ids) and torch.equal(r.loss, r2.loss)
    assert torch.equal(d, nsp.distill_grad(x, top, ids)[1])


def refused(nsp, call):
    with pytest.raises(nsp.NsPackError) as e:
        call()
    assert e.value.code == nsp.NS_ERR_INVALID_ARG


def test_scan_refusals(nsp):
    z = torch.randn(2, 5, 8).cuda()
    i = torch.zeros(2, 5, dtype=torch.int32).cuda()
    b = torch.zeros(8).cuda()
    for call in (
            lambda: nsp.gated_scan(z.cpu(), z), lambda: nsp.gated_scan(z, z.cpu()),
            lambda: nsp.gated_scan(z.double(), z.double()), lambda: nsp.gated_scan(z, z.half()),
            lambda: nsp.gated_scan(z[0], z[0]), lambda: nsp.gated_scan(z, z[:, :4]),
            lambda: nsp.gated_scan(z.transpose(1, 2), z.transpose(1, 2)),
            lambda: nsp.gated_scan(z, None), lambda: nsp.gated_scan(z, z, b[:7]),
            lambda: nsp.gated_scan(z, z, b.half()), lambda: nsp.gated_scan(z, z, b.cpu()),
            lambda: nsp.gated_scan(z, z, pos=i.long()), lambda: nsp.gated_scan(z, z, doc=i[:, :4]),
            lambda: nsp.gated_scan(z, z, pos=i.t().contiguous().t()),
            lambda: nsp.gated_scan(z, z, h0=z[:, 0].half()), lambda: nsp.gated_scan(z, z, h0=b)):
        refused(nsp, call)
    y, h, st = nsp.gated_scan_forward(z, z)
    for call in (
            lambda: nsp.gated_scan_backward(y[:, :4], h, z, z, None, st),
            lambda: nsp.gated_scan_backward(y.half(), h, z, z, None, st),
            lambda: nsp.gated_scan_backward(y, h, z, z, None, None),
            lambda: nsp.gated_scan_backward(y, h, z, z, None, st[:, :0]),
            lambda: nsp.gated_scan_backward(y, h[:1], z, z, None, st)):
        refused(nsp, call)


def test_distill_refusals(nsp):
    x = torch.randn(4, 50).cuda()
    top, ids = x.topk(3, 1)
    w = torch.ones(4).cuda()
    long = torch.zeros(4, 1025, dtype=torch.int32).cuda()
    for call in (
            lambda: nsp.distill_loss(x.cpu(), top, ids), lambda: nsp.distill_loss(x[0], top, ids),
            lambda: nsp.distill_loss(x.t(), top, ids), lambda: nsp.distill_loss(x.double(), top, ids),
            lambda: nsp.distill_loss(x, top[:3], ids), lambda: nsp.distill_loss(x, top, ids[:, :2]),
            lambda: nsp.distill_loss(x, top, ids.short()), lambda: nsp.distill_loss(x, top, None),
            lambda: nsp.distill_loss(x, top[:, :0], ids[:, :0]),
            lambda: nsp.distill_loss(x, long.float(), long),
            lambda: nsp.distill_loss(x, top, ids, mask=w),
            lambda: nsp.distill_loss(x, top, ids, mask=torch.ones(3).byte().cuda()),
            lambda: nsp.distill_loss(x, top, ids, temperature=0.0),
            lambda: nsp.distill_loss(x, top, ids, temperature=-1.0),
            lambda: nsp.distill_loss(x, top, ids, temperature=NAN),
            lambda: nsp.distill_loss(x, top, ids, temperature=INF),
            lambda: nsp.distill_loss(x, top, ids, temperature=1e-39),
            lambda: nsp.distill_loss(x, top, ids, teacher_lse=w.half()),
            lambda: nsp.distill_grad(x, top, ids, weight=w[:3]),
            lambda: nsp.distill_grad(x, top, ids, weight=w.cpu()),
            lambda: nsp.distill_grad(x, top, ids, out=x.half()),
            lambda: nsp.distill_grad(x, top, ids, out=x[:, :40]),
            lambda: nsp.distill_grad(x[:, :25], top, ids, out=x[:, 20:45]),  # overlaps in part
            lambda: nsp.distill_grad(x.expand(4, 50)[:1].expand(4, 50), top, ids)):
        refused(nsp, call)


def test_route_refusals(nsp):
    x = torch.randn(6, 40).cuda()
    r = nsp.route(x, 4)
    dw = torch.ones(6, 4).cuda()
    big = torch.randn(2, 1025).cuda()
    for call in (
            lambda: nsp.route(x.cpu(), 4), lambda: nsp.route(x[0], 4), lambda: nsp.route(x, 0),
            lambda: nsp.route(x, 41), lambda: nsp.route(x, 33), lambda: nsp.route(x, -1),
            lambda: nsp.route(x, 2.0), lambda: nsp.route(x.double(), 4), lambda: nsp.route(x.t(), 4),
            lambda: nsp.route(big, 4), lambda: nsp.route(x, 4, doc=torch.zeros(6).cuda()),
            lambda: nsp.route(x, 4, doc=torch.zeros(5, dtype=torch.int32).cuda()),
            lambda: nsp.route(x[:, :0], 1),
            lambda: nsp.route_backward(x, r, dw[:, :3]), lambda: nsp.route_backward(x, r, dw.half()),
            lambda: nsp.route_backward(x, None, dw), lambda: nsp.route_backward(x[:, :39], r, dw),
            lambda: nsp.route_backward(x, r, dw, torch.ones(2).cuda())):
        refused(nsp, call)


def test_operators_on_a_packed_update(nsp):
    """The packer's own arrays through every operator, forward and backward, by the
    example: the loss falls, and padding chose no expert."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "packed_training_step.py")
    spec = importlib.util.spec_from_file_location("packed_training_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=8)
    assert all(math.isfinite(x) for x in losses) and losses[-1] < losses[0] - 0.1
    from corpus import make_preset
    c = make_preset("c1")
    pk = nsp.Packer.from_corpus(c)
    out = pk.step(0)
    doc = out["doc"][0]
    r = nsp.route(torch.randn(doc.numel(), 8, generator=gen(1)).cuda(), 2, doc=doc.reshape(-1))
    assert int(r.tokens) == int((doc >= 0).sum())
    assert ((r.ids == -1).all(1) == (doc.reshape(-1) < 0)).all()
    # packed rows give what their documents give alone
    z = torch.randn(*doc.shape, 32, generator=gen(2)).cuda()
    f = torch.randn(*doc.shape, 32, generator=gen(3)).cuda()
    y, _ = nsp.gated_scan(z, f, pos=out["pos"][0], doc=doc)
    row, pos = doc[0].cpu(), out["pos"][0][0].cpu()
    starts = [t for t in range(len(row)) if pos[t] == 0 and row[t] >= 0] + [int((row >= 0).sum())]
    for a, b in zip(starts[:6], starts[1:7]):
        alone, _ = nsp.gated_scan(z[:1, a:b], f[:1, a:b])
        close(y[0, a:b], alone[0].double().cpu(), 2e-5, f"document at {a}")
    pk.close()

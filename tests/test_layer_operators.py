"""The kernels of embed, layer_norm, dispatch and combine against plain 64-bit forms of
their formulas.

Tolerances are bounds, element by element, with u = 2**-24 the rounding of a 32-bit
float and a 16-bit output's own rounding (2**-8 or 2**-11 of the value, half a step
among the smallest):

* a sum of n terms in any order is off by at most n u times the sum of their sizes;
* a row's sums go through at most 80 values a lane, 5 steps among lanes and 16 among
  warps, and twice the bound of that covers the few roundings around them: C = 256 (rows
  that are not kept: D / 4096 chunks of 8 a lane, no more for the widths here).  With A =
  mean |x| / sigma the normalised value xh is off by e = C u (A + |xh|), and dx = r (g - mean
  g - xh mean(g xh)) by r C u (|g| + 2 G + |xh| (G A + 3 M) + A M) + C u |dx|, where G =
  mean |g| and M = mean |g xh|.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
LEAST = {torch.float32: 2.0**-149, torch.bfloat16: 2.0**-133, torch.float16: 2.0**-24}
U, C = 2.0**-24, 256
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


def within(got, want, tol, name):
    """|got - want| <= tol and the output's own rounding, and NaN in the same places."""
    dt = got.dtype
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    tol = torch.as_tensor(tol, dtype=torch.float64) + ROUND[dt] * 1.01 * want.abs() + LEAST[dt]
    off = (got - want).abs() - tol
    off = off[~torch.isnan(want)]
    assert off.numel() == 0 or float(off.max()) <= 0.0, (name, float(off.max()))


def same(a, b):
    assert a.shape == b.shape and a.dtype == b.dtype
    flat = (lambda t: t.contiguous().view(-1).view(torch.uint8))
    return torch.equal(flat(a), flat(b))


def laid(t, pad=0, shift=0):
    """A copy on the GPU whose rows are `pad` elements apart, `shift` off a boundary."""
    D = t.shape[-1]
    rows = t.numel() // D if D else 0
    flat = torch.full((rows * (D + pad) + shift + 1,), NAN, dtype=t.dtype, device="cuda")
    out = flat[shift:shift + rows * (D + pad)].view(*t.shape[:-1], D + pad)[..., :D]
    return out.copy_(t)


# ---- rows of a table ---------------------------------------------------------------
def check_embed(nsp, weight, tokens, doc, scale, out_dtype, dy, weight_cuda=None, dy_cuda=None):
    V, D = weight.shape
    s = float(torch.tensor(scale, dtype=torch.float32))
    real = (tokens >= 0) & (tokens < V)
    if doc is not None:
        real &= doc >= 0
    at = torch.where(real, tokens, torch.zeros_like(tokens)).long()
    want = torch.zeros(*tokens.shape, D, dtype=torch.float64)
    if V:
        want = torch.where(real[..., None], weight.double()[at] * s, want)
    wc = weight.cuda() if weight_cuda is None else weight_cuda
    kw = dict(scale=scale, doc=dev(doc))
    y = nsp.embed(wc, tokens.cuda(), dtype=out_dtype, **kw)
    within(y, want, 2 * U * want.abs(), "y")
    if dy is None:
        return
    flat, ids = dy.double().reshape(-1, D), at.reshape(-1)
    flat = torch.where(real.reshape(-1)[:, None], flat, torch.zeros_like(flat))
    total = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids, flat)
    sizes = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids, flat.abs())
    count = torch.zeros(V, dtype=torch.float64).index_add_(0, ids, real.reshape(-1).double())
    d = nsp.embed_backward(dy.cuda() if dy_cuda is None else dy_cuda, tokens.cuda(), V,
                           dtype=weight.dtype, **kw)
    within(d, total * s, (count[:, None] + 2) * U * sizes * abs(s), "dweight")
    assert (d[(count == 0).cuda()] == 0).all()


@pytest.mark.parametrize("wtype,dtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                         ("f32", "bf16"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("N,V,D", [
    (1, 1, 1), (5, 3, 2), (33, 7, 8), (64, 100, 64), (70, 511, 65), (300, 512, 31), (257, 600, 257),
    (1000, 50, 264), (31, 2000, 1001), (2049, 70000, 40), (700, 300000, 24), (4100, 9, 519)])
def test_embed(nsp, N, V, D, wtype, dtype):
    g = gen(N + V + D)
    weight = torch.randn(V, D, generator=g).to(DTYPES[wtype])
    tokens = (torch.rand(N, generator=g) ** 3 * V).int()
    doc = (torch.rand(N, generator=g) < 0.9).int() - 1
    dy = torch.randn(N, D, generator=g).to(DTYPES[dtype])
    check_embed(nsp, weight, tokens, doc, 1.7, DTYPES[dtype], dy)
    check_embed(nsp, weight, tokens.long(), None, 1.0, DTYPES[dtype], dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (16, 4), (1, 2)])
def test_embed_strides_and_alignment(nsp, pad, shift, dtype):
    for D in (40, 39, 520, 1):
        g = gen(D + pad)
        weight = torch.randn(90, D, generator=g).to(DTYPES[dtype])
        tokens = (torch.rand(3, 150, generator=g) ** 2 * 90).int()
        dy = torch.randn(3, 150, D, generator=g).to(DTYPES[dtype])
        check_embed(nsp, weight, tokens, None, 0.5, DTYPES[dtype], dy, laid(weight, pad, shift),
                    laid(dy, pad, shift))


def test_embed_runs_of_every_length_at_every_place(nsp):
    """Tokens of 1 to 100 positions one after the other in the sorted order, so that they
    begin, end and go on at the tiles' edges in all ways; and one token alone."""
    g = gen(5)
    lengths = list(range(1, 101)) + [32] * 5 + [31, 33, 1, 64, 63, 65, 1, 31, 1000, 31, 2, 97]
    tokens = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(lengths)])
    perm = torch.randperm(len(tokens), generator=g)
    for dtype, D in (("f32", 33), ("bf16", 72), ("bf16", 300), ("f16", 71)):
        dy = torch.randn(len(tokens), D, generator=g).to(DTYPES[dtype])
        w = torch.randn(len(lengths), D, generator=g).to(DTYPES[dtype])
        check_embed(nsp, w, tokens[perm], None, 1.0, None, dy)
        for n in (31, 32, 33, 63, 64, 65, 3001):
            check_embed(nsp, w, torch.full((n,), 7, dtype=torch.int32), None, 1.0, None,
                        dy[:1].expand(n, D).clone())


def test_embed_many_positions(nsp):
    g = gen(8)
    for N, V, D in ((130_001, 700, 16), (90_000, 50257, 9)):
        tokens = (torch.rand(N, generator=g) ** 4 * V).int()
        dy = torch.randn(N, D, generator=g)
        check_embed(nsp, torch.randn(V, D, generator=g), tokens, None, 1.0, None, dy)


def test_embed_tokens_outside_and_padding(nsp):
    w = torch.randn(10, 12, generator=gen(1))
    tokens = torch.tensor([0, -1, 9, 10, 2**31 - 1, -2**31, 3, 3, 5, 0])
    doc = torch.tensor([0, 0, 0, 0, 0, 0, -1, 4, -2**31, 2**31 - 1]).int()
    dy = torch.randn(10, 12, generator=gen(2))
    check_embed(nsp, w, tokens.int(), doc, 2.0, None, dy)
    tokens[4], tokens[5] = 2**40 + 3, -2**40  # what is left of them in 32 bits is a token
    check_embed(nsp, w, tokens, doc, 2.0, None, dy)
    gone = (doc < 0) | (tokens < 0) | (tokens >= 10)
    want = nsp.embed_backward(dy.cuda(), tokens.cuda(), 10, doc=doc.cuda())
    for bad in (NAN, INF, -INF):
        d = torch.where(gone[:, None], torch.full_like(dy, bad), dy)
        assert same(nsp.embed_backward(d.cuda(), tokens.cuda(), 10, doc=doc.cuda()), want)
    # a NaN reaches its own token's row alone
    dy[0, 3] = NAN
    d = nsp.embed_backward(dy.cuda(), tokens.cuda(), 10, doc=doc.cuda())
    assert torch.isnan(d[0, 3]) and not torch.isnan(d).any(1)[1:].any()
    # all of it padding
    none = torch.full((10,), -1, dtype=torch.int32).cuda()
    assert (nsp.embed(w.cuda(), tokens.cuda(), doc=none) == 0).all()
    assert (nsp.embed_backward(dy.cuda(), tokens.cuda(), 10, doc=none) == 0).all()


def test_embed_of_nothing(nsp):
    w = torch.randn(6, 5).cuda()
    t = torch.zeros(0, 3, dtype=torch.int32).cuda()
    assert nsp.embed(w, t).shape == (0, 3, 5)
    assert torch.equal(nsp.embed_backward(torch.zeros(0, 3, 5).cuda(), t, 6), torch.zeros_like(w))
    t = torch.zeros(4, dtype=torch.int64).cuda()
    assert (nsp.embed(w[:0], t) == 0).all()
    assert nsp.embed_backward(torch.zeros(4, 5).cuda(), t, 0).shape == (0, 5)
    assert nsp.embed(w[:, :0], t).shape == (4, 0)
    assert nsp.embed(w, t[0]).shape == (5,)


def test_embed_offsets_past_32_bits(nsp):
    N, D, V = 1_050_000, 2056, 1_048_600  # over 2**31 elements of y, dy and the table
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[-1], w[5] = 3.0, 2.0
    tokens = torch.full((N,), 5, dtype=torch.int32, device="cuda")
    tokens[::2] = torch.arange(N // 2, device="cuda", dtype=torch.int32)
    tokens[-1] = V - 1
    y = nsp.embed(w, tokens)
    assert (y[-1] == 3).all() and (y[1::2][:-1] == 2).all() and (y[N - 2] == 0).all()
    del w
    y.zero_()
    y[-1], y[-3], y[1] = 4.0, 1.0, 0.5
    d = nsp.embed_backward(y, tokens, V)
    assert (d[-1] == 4).all() and (d[5] == 1.5).all()
    d[-1], d[5] = 0, 0
    assert not d.any()


def test_embed_gradient_and_autograd(nsp):
    g = gen(11)
    w = torch.randn(40, 24, generator=g).cuda().requires_grad_()
    tokens = torch.randint(0, 44, (3, 50), generator=g).int().cuda()
    doc = ((torch.rand(3, 50, generator=g) < 0.9).int() - 1).cuda()
    c = torch.randn(3, 50, 24, generator=g).cuda()

    def value(x):
        return (nsp.embed(x, tokens, scale=1.5, doc=doc).double() * c.double()).sum()

    (grad,) = torch.autograd.grad(value(w), w)
    assert same(grad, nsp.embed_backward(c, tokens, 40, scale=1.5, doc=doc))
    # it is linear: differences are off by the roundings of values alone
    v = torch.randn(40, 24, generator=g).cuda()
    slope = float((grad.double() * v.double()).sum())
    with torch.no_grad():
        got = float(value(w + v) - value(w - v)) / 2
    assert abs(got - slope) <= 1e-4 * float((grad.double() * v.double()).abs().sum())
    # gradients that are laid out otherwise: broadcast, transposed, of one column
    for lay in (lambda y: y.sum(), lambda y: y.transpose(0, 1).contiguous().view(-1)[::3].sum(),
                lambda y: (y[..., 0] * 2).sum(), lambda y: y[:, ::2].sum()):
        (a,) = torch.autograd.grad(lay(nsp.embed(w, tokens, doc=doc)), w)
        y = nsp.embed(w, tokens, doc=doc).detach().requires_grad_()
        (dy,) = torch.autograd.grad(lay(y), y)
        assert same(a, nsp.embed_backward(dy.contiguous(), tokens, 40, doc=doc))
    (a,) = torch.autograd.grad(nsp.embed(w, tokens, dtype=torch.bfloat16).float().sum(), w)
    assert a.dtype == torch.float32


# ---- layer norm ------------------------------------------------------------------------
def norm_reference(x, w, b, eps, doc, dy=None):
    """Values and the bounds of their errors."""
    D = x.shape[-1]
    x = x.double()
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(D, dtype=torch.float64) if b is None else b.double()
    gone = torch.zeros(x.shape[:-1], dtype=torch.bool) if doc is None else doc < 0
    x = torch.where(gone[..., None], torch.zeros_like(x), x)
    mean = x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mean) * r
    A = x.abs().mean(-1, keepdim=True) * r
    e = C * U * (A + xh.abs())
    zero = torch.zeros_like(x)
    keep = (lambda t: torch.where(gone[..., None], zero, t))
    y = xh * w + b
    out = dict(y=keep(y), y_tol=w.abs() * e + 3 * U * ((xh * w).abs() + b.abs()))
    if dy is None:
        return out
    dy = keep(dy.double())
    g = dy * w
    s1, s2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = r * (g - s1 - xh * s2)
    G, M = g.abs().mean(-1, keepdim=True), (g * xh).abs().mean(-1, keepdim=True)
    out.update(dx=keep(dx), dx_tol=r * C * U * (g.abs() + 2 * G + xh.abs() * (G * A + 3 * M) + A * M)
               + C * U * dx.abs())
    lead = tuple(range(x.dim() - 1))
    n = x.numel() // D + 64
    out.update(dw=(dy * xh).sum(lead), db=dy.sum(lead),
               dw_tol=(dy.abs() * e).sum(lead) + n * U * (dy * xh).abs().sum(lead),
               db_tol=n * U * dy.abs().sum(lead))
    return out


def check_norm(nsp, x, w, b, doc, dy, eps=1e-5, xc=None, dyc=None, wc=None, bc=None):
    want = norm_reference(x, w, b, eps, doc, dy)
    xc = x.cuda() if xc is None else xc
    dyc = dy.cuda() if dyc is None else dyc
    wc, bc = dev(w) if wc is None else wc, dev(b) if bc is None else bc
    y, mean, rstd = nsp.layer_norm_forward(xc, wc, bc, eps=eps, doc=dev(doc))
    assert same(y, nsp.layer_norm(xc, wc, bc, eps=eps, doc=dev(doc)))
    within(y, want["y"], want["y_tol"], "y")
    dx, dw, db = nsp.layer_norm_backward(dyc, xc, wc, bc, mean, rstd, doc=dev(doc))
    within(dx, want["dx"], want["dx_tol"], "dx")
    assert (dw is None) == (w is None) and (db is None) == (b is None)
    if w is not None:
        within(dw, want["dw"], want["dw_tol"], "dweight")
    if b is not None:
        within(db, want["db"], want["db_tol"], "dbias")


def norm_inputs(N, D, dtype, wtype, seed):
    g = gen(seed)
    dt = DTYPES[dtype]
    x = (torch.randn(N, D, generator=g) * (torch.rand(N, 1, generator=g) * 4 + 0.1)
         + torch.randn(N, 1, generator=g)).to(dt)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(DTYPES[wtype])
    b = (0.3 * torch.randn(D, generator=g)).to(DTYPES[wtype])
    doc = (torch.rand(N, generator=g) < 0.85).int() - 1
    return x, w, b, doc, torch.randn(N, D, generator=g).to(dt)


@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                         ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("N,D", [
    (1, 1), (3, 2), (70, 7), (5, 8), (33, 9), (9, 16), (40, 31), (100, 64), (33, 65), (20, 127),
    (17, 128), (9, 255), (64, 256), (7, 257), (11, 511), (5, 520), (30, 1001), (12, 1280),
    (3, 2047), (600, 40), (5, 2560), (4, 2571), (3, 4099), (2, 5003), (3, 8192), (2, 8200),
    (2, 8193), (1, 20481), (2, 41000)])
def test_layer_norm(nsp, N, D, dtype, wtype):
    x, w, b, doc, dy = norm_inputs(N, D, dtype, wtype, N + D)
    check_norm(nsp, x, w, b, doc, dy)
    if wtype == "f32":
        check_norm(nsp, x, w, None, None, dy)
    elif D % 3 == 0:
        check_norm(nsp, x, None, b, doc, dy)
    else:
        check_norm(nsp, x, None, None, doc, dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(5_001, 96), (3_003, 513), (2_111, 1280), (70_001, 12),
                                 (301, 9000)])
def test_layer_norm_many_rows(nsp, N, D, dtype):
    x, w, b, doc, dy = norm_inputs(N, D, dtype, "f32", D)
    check_norm(nsp, x, w, b, doc, dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,D", [(2500, 514), (1300, 1281), (1001, 2560), (701, 2571), (650, 3841),
                                 (640, 5003), (630, 7682), (620, 8200), (613, 11521), (611, 16384),
                                 (610, 19200)])
def test_layer_norm_rows_through_the_ring(nsp, N, D, dtype):
    """Enough rows for every width of row, and of pieces, to come through shared memory, in
    batches of which the last is not whole; padding of whole batches; the rows' places an odd
    distance apart, and off a boundary."""
    x, w, b, doc, dy = norm_inputs(N, D, dtype, "f32", N + D)
    doc[40:80] = -1
    doc[-1] = 0
    check_norm(nsp, x, w, b, doc, dy)
    if dtype != "f16":
        check_norm(nsp, x, w, b, None, dy, xc=laid(x, 3, 5), dyc=laid(dy, 1, 7))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (16, 4), (1, 2), (5, 7)])
def test_layer_norm_strides_and_alignment(nsp, pad, shift, dtype):
    for N, D in ((40, 64), (40, 63), (7, 519), (6, 1301), (5, 2600), (3, 8300)):
        x, w, b, doc, dy = norm_inputs(N, D, dtype, dtype, D + pad)
        check_norm(nsp, x, w, b, doc, dy, xc=laid(x, pad, shift), dyc=laid(dy, shift, pad % 8),
                   wc=laid(w, 0, shift), bc=laid(b, 0, pad))
    x, w, b, doc, dy = norm_inputs(60, 48, dtype, "f32", pad)
    x3, dy3, doc3 = x.view(3, 20, 48), dy.view(3, 20, 48), doc.view(3, 20)
    check_norm(nsp, x3, w, b, doc3, dy3, xc=laid(x3, pad, shift), dyc=laid(dy3, pad, shift))


@pytest.mark.parametrize("D", [24, 100, 1280, 8200])
def test_layer_norm_extreme_rows(nsp, D):
    g = gen(D)
    x = torch.randn(8, D, generator=g)
    x[1] += 1e4            # a mean far from 0
    x[2] = 3.0             # constant: only eps is left
    x[3] *= 1e15
    x[4] *= 1e-12
    x[5] = 0
    x[6, 0] = 1e6          # one channel alone
    w, b = torch.randn(D, generator=g), torch.randn(D, generator=g)
    dy = torch.randn(8, D, generator=g)
    check_norm(nsp, x, w, b, None, dy)
    check_norm(nsp, x[[0, 1, 3, 6, 7]], w, b, None, dy[:5], eps=0.0)


@pytest.mark.parametrize("D", [5, 64, 513, 2560, 8200])
def test_layer_norm_padding_is_not_read_and_nan_stays_in_its_row(nsp, D):
    x, w, b, doc, dy = norm_inputs(40, D, "f32", "f32", D)
    doc[7], doc[8] = -1, 0
    args = (w.cuda(), b.cuda())
    y, m, r = nsp.layer_norm_forward(x.cuda(), *args, doc=doc.cuda())
    want = nsp.layer_norm_backward(dy.cuda(), x.cuda(), *args, m, r, doc=doc.cuda())
    assert (y[(doc < 0).cuda()] == 0).all() and (want[0][(doc < 0).cuda()] == 0).all()
    for bad in (NAN, INF, torch.finfo(torch.float32).min):
        xb = torch.where((doc < 0)[:, None], torch.full_like(x, bad), x).cuda()
        db = torch.where((doc < 0)[:, None], torch.full_like(x, bad), dy).cuda()
        y2, m2, r2 = nsp.layer_norm_forward(xb, *args, doc=doc.cuda())
        assert same(y, y2) and same(m, m2) and same(r, r2)
        m2[7], r2[7] = NAN, NAN
        got = nsp.layer_norm_backward(db, xb, *args, m2, r2, doc=doc.cuda())
        for a, c in zip(got, want):
            assert same(a, c)
    x[8, D // 2] = NAN
    y2 = nsp.layer_norm(x.cuda(), *args, doc=doc.cuda())
    rows = torch.arange(40) != 8
    assert torch.isnan(y2[8]).all() and same(y2[rows.cuda()], y[rows.cuda()])
    none = torch.full((40,), -1, dtype=torch.int32).cuda()
    y2, m, r = nsp.layer_norm_forward(x.cuda(), *args, doc=none)
    got = nsp.layer_norm_backward(dy.cuda(), x.cuda(), *args, m, r, doc=none)
    assert not any(t.any() for t in (y2, m, r, *got))


def test_layer_norm_of_nothing(nsp):
    x = torch.zeros(0, 4, 6).cuda()
    w = torch.ones(6).cuda()
    y, m, r = nsp.layer_norm_forward(x, w, w)
    assert y.shape == (0, 4, 6)
    dx, dw, db = nsp.layer_norm_backward(x, x, w, w, m, r)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
    x = torch.zeros(0, 9000).cuda()
    w = torch.ones(9000).cuda()
    y, m, r = nsp.layer_norm_forward(x, w, w)
    assert not nsp.layer_norm_backward(x, x, w, w, m, r)[1].any()


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (300, "f16"), (520, "f32"), (1001, "bf16"),
                                     (2560, "bf16"), (4096, "f32"), (5003, "bf16"), (8192, "f16"),
                                     (16384, "bf16")])
def test_layer_norm_rows_do_not_depend_on_the_other_rows(nsp, D, dtype):
    x, w, b, doc, dy = (t.cuda() for t in norm_inputs(700, D, dtype, "f32", D))
    y, m, r = nsp.layer_norm_forward(x, w, b, doc=doc)
    dx = nsp.layer_norm_backward(dy, x, w, b, m, r, doc=doc)[0]
    for rows in (slice(3, 4), slice(17, 60)):
        y1, m1, r1 = nsp.layer_norm_forward(x[rows], w, b, doc=doc[rows])
        assert same(y1, y[rows]) and same(m1, m[rows]) and same(r1, r[rows])
        assert same(nsp.layer_norm_backward(dy[rows], x[rows], w, b, m1, r1, doc=doc[rows])[0],
                    dx[rows])


def test_layer_norm_offsets_past_32_bits(nsp):
    N, D = 1_050_000, 2056
    x = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    x[-1, ::2], x[-1, 1::2] = 1.0, -1.0
    y, m, r = nsp.layer_norm_forward(x)
    assert (y[-1] == x[-1]).all() and not y[:-1].any()
    dx, _, db = nsp.layer_norm_backward(x, x, None, torch.zeros(D).cuda(), m, r)
    assert not dx[:-1].any() and float(dx[-1].float().abs().max()) < 1e-2
    assert torch.equal(db, x[-1].float())


def directional(value, x, v, step):
    return (value(x + step * v) - value(x - step * v)) / (2 * step)


def test_layer_norm_gradients_against_differences(nsp):
    """Central differences of an O(1) function: of step 2e-2 off by some 4e-4 of it, and by
    the roundings of 32 bits, 1e-7 / 2e-2 of the sum of the terms' sizes."""
    x, w, b, doc, dy = (t.cuda() for t in norm_inputs(30, 40, "f32", "f32", 4))
    x = x / x.std(1, keepdim=True)

    def value(x, w, b):
        y = nsp.layer_norm(x, w, b, doc=doc)
        return (y.double() * dy.double()).sum()

    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    grads = torch.autograd.grad(value(*leaves), leaves)
    y, m, r = nsp.layer_norm_forward(x, w, b, doc=doc)
    for a, e in zip(grads, nsp.layer_norm_backward(dy, x, w, b, m, r, doc=doc)):
        assert same(a, e)
    sizes = float((y.double() * dy.double()).abs().sum())
    for i, t in enumerate((x, w, b)):
        v = grads[i] / grads[i].abs().max()
        slope = float((grads[i].double() * v.double()).sum())
        args = [x, w, b]

        def f(z):
            args[i] = z
            return float(value(*args))

        got = directional(f, t, v, 2e-2)
        assert abs(got - slope) <= 5e-3 * abs(slope) + 1e-5 * sizes, i


def test_layer_norm_autograd(nsp):
    x, w, b, doc, dy = (t.cuda() for t in norm_inputs(24, 40, "bf16", "f32", 3))
    x = x.view(4, 6, 40).requires_grad_()
    w.requires_grad_()
    for lay in (lambda y: y.float().sum(), lambda y: (y[:, ::2].float() * 2).sum(),
                lambda y: y.transpose(0, 1).reshape(-1)[::7].float().sum()):
        y = nsp.layer_norm(x, w, b, doc=doc.view(4, 6))
        dx, dw = torch.autograd.grad(lay(y), (x, w))
        z = y.detach().requires_grad_()
        (dz,) = torch.autograd.grad(lay(z), z)
        _, m, r = nsp.layer_norm_forward(x.detach(), w.detach(), b, doc=doc.view(4, 6))
        e = nsp.layer_norm_backward(dz.contiguous(), x.detach(), w.detach(), b, m, r,
                                    doc=doc.view(4, 6))
        assert same(dx, e[0]) and same(dw, e[1])


# ---- tokens by expert, and back ---------------------------------------------------------
def expert_reference(x, ids, E):
    N, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    slots = torch.tensor(sorted(range(N * k), key=lambda s: (int(key[s]), s)), dtype=torch.long)
    place = torch.empty(N * k, dtype=torch.long)
    place[slots] = torch.arange(N * k)
    offsets = torch.tensor([int((key < e).sum()) for e in range(E + 1)])
    rows = torch.where((key[slots] < E)[:, None], x[slots // k], torch.zeros_like(x[slots // k]))
    return place.view(N, k), slots, offsets, rows, (key < E).view(N, k)


def check_experts(nsp, x, ids, E, y, w, d_out, pad=0, shift=0):
    N, k = ids.shape
    place, slots, offsets, rows, there = expert_reference(x, ids, E)
    got, order = nsp.dispatch(laid(x, pad, shift) if pad or shift else x.cuda(), ids.cuda(), E)
    for a, b, name in zip(order, (place, slots, offsets), ("place", "slots", "offsets")):
        assert torch.equal(a.cpu().long(), b), name
    assert same(got.cpu(), rows)
    yc = laid(y, pad, shift) if pad or shift else y.cuda()
    dc = laid(d_out, pad, shift) if pad or shift else d_out.cuda()
    each = torch.where(there[..., None], y.double()[place], torch.zeros(1, dtype=torch.float64))
    out = nsp.combine(yc, order, w.cuda())
    terms = w.double()[..., None] * each
    within(out, terms.sum(1), (k + 1) * U * terms.abs().sum(1), "out")
    plain = nsp.combine(yc, order)
    within(plain, each.sum(1), k * U * each.abs().sum(1), "out without weights")
    assert same(nsp.dispatch_backward(yc, order), plain)
    d_rows, d_w = nsp.combine_backward(dc, yc, order, w.cuda())
    want = torch.zeros(N * k, x.shape[1], dtype=torch.float64)
    want[place.view(-1)] = (torch.where(there, w, torch.zeros_like(w)).double()[..., None]
                            * d_out.double()[:, None]).view(N * k, -1)
    within(d_rows, want, U * want.abs(), "d_rows")
    assert (d_rows[int(offsets[E]):] == 0).all()
    dots = each * d_out.double()[:, None]
    within(d_w, dots.sum(2), (x.shape[1] + 16) * U * dots.abs().sum(2), "d_weights")
    d_rows, none = nsp.combine_backward(dc, yc, order)
    assert none is None and torch.equal(d_rows.cpu()[place[there]],
                                        d_out[:, None].expand(N, k, -1)[there])


def expert_inputs(N, E, k, D, dtype, seed, gone=0.1):
    g = gen(seed)
    dt = DTYPES[dtype]
    ids = (torch.rand(N, k, generator=g) ** 2 * E).int()
    ids[torch.rand(N, k, generator=g) < gone] = -1
    return (torch.randn(N, D, generator=g).to(dt), ids, E, torch.randn(N * k, D, generator=g).to(dt),
            torch.rand(N, k, generator=g), torch.randn(N, D, generator=g).to(dt))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,E,k,D", [
    (1, 1, 1, 1), (3, 2, 1, 2), (64, 64, 8, 64), (7, 5, 3, 9), (33, 8, 2, 31), (256, 8, 8, 40),
    (257, 8, 8, 40), (100, 1024, 4, 65), (700, 1024, 4, 24), (2048, 3, 1, 16), (2049, 3, 1, 15),
    (300, 60, 5, 513), (50, 16, 33, 8), (9, 300, 100, 257), (1500, 256, 3, 260), (5, 4, 2, 2571)])
def test_experts(nsp, N, E, k, D, dtype):
    check_experts(nsp, *expert_inputs(N, E, k, D, dtype, N + E + k + D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (16, 4), (1, 2)])
def test_experts_strides_and_alignment(nsp, pad, shift, dtype):
    for N, D in ((40, 64), (40, 63), (900, 40), (700, 519)):
        check_experts(nsp, *expert_inputs(N, 10, 4, D, dtype, D + pad), pad, shift)


@pytest.mark.parametrize("N", [60, 5000])
def test_experts_masks(nsp, N):
    """Every choice without an expert, none, one expert alone, the same expert twice for a
    token, ids out of range."""
    x, ids, E, y, w, d = expert_inputs(N, 6, 3, 20, "f32", N)
    for fill in (-1, 0, 5, 6, 2**31 - 1, -2**31):
        check_experts(nsp, x, torch.full_like(ids, fill), E, y, w, d)
    ids[:, 1] = ids[:, 0]
    ids[::7, 2] = 77
    ids[3] = -1
    check_experts(nsp, x, ids, E, y, w, d)


@pytest.mark.parametrize("N,E,k", [(40_000, 64, 8), (100_003, 7, 2), (30_000, 1024, 3)])
def test_experts_many_tokens(nsp, N, E, k):
    g = gen(N)
    ids = (torch.rand(N, k, generator=g) ** 2 * (E + 1)).int().cuda()
    x = torch.randn(N, 8, generator=g).cuda()
    rows, order = nsp.dispatch(x, ids, E)
    key = torch.where((ids >= 0) & (ids < E), ids, E).view(-1)
    slots = torch.sort(key, stable=True).indices
    assert torch.equal(order.slots.long(), slots)
    assert torch.equal(order.place.view(-1)[slots].long(), torch.arange(N * k, device="cuda"))
    assert torch.equal(order.offsets.long(),
                       torch.searchsorted(key[slots], torch.arange(E + 1, device="cuda").int()))
    assert torch.equal(rows, x[slots // k] * (key[slots] < E)[:, None])


def test_experts_keep_what_16_bits_hold(nsp):
    # rows are moved as they are: NaN, infinities, zeros of both signs, subnormal numbers
    bits = torch.arange(-2**15, 2**15, dtype=torch.int32).to(torch.int16).view(64, 1024)
    ids = torch.randint(0, 9, (64, 3), generator=gen(0)).int()
    for dt in (torch.bfloat16, torch.float16):
        rows, order = nsp.dispatch(bits.view(dt).cuda(), ids.cuda(), 9)
        assert torch.equal(rows.view(torch.int16)[order.place.view(-1).long()].cpu(),
                           bits.repeat_interleave(3, 0))


def test_experts_rows_without_a_choice_are_not_read(nsp):
    x, ids, E, y, w, d = expert_inputs(50, 4, 3, 24, "f32", 2, gone=0.5)
    _, order = nsp.dispatch(x.cuda(), ids.cuda(), E)
    M = int(order.offsets[E])
    y2, w2 = y.clone(), torch.where(ids < 0, torch.full_like(w, NAN), w)
    y2[M:] = NAN
    assert same(nsp.combine(y.cuda(), order, w.cuda()), nsp.combine(y2.cuda(), order, w2.cuda()))
    for a, b in zip(nsp.combine_backward(d.cuda(), y.cuda(), order, w.cuda()),
                    nsp.combine_backward(d.cuda(), y2.cuda(), order, w2.cuda())):
        assert same(a, b)
    assert same(nsp.dispatch_backward(y.cuda(), order), nsp.dispatch_backward(y2.cuda(), order))


def test_experts_of_nothing(nsp):
    x = torch.zeros(0, 5).cuda()
    ids = torch.zeros(0, 2, dtype=torch.int32).cuda()
    rows, order = nsp.dispatch(x, ids, 3)
    assert rows.shape == (0, 5) and torch.equal(order.offsets.cpu(), torch.zeros(4).int())
    assert nsp.combine(rows, order).shape == (0, 5)
    assert nsp.combine_backward(x, rows, order, torch.zeros(0, 2).cuda())[1].shape == (0, 2)
    for N in (4, 3000):
        x = torch.zeros(N, 0).cuda()
        ids = torch.zeros(N, 2, dtype=torch.int32).cuda()
        rows, order = nsp.dispatch(x, ids, 3)
        assert order.offsets.tolist() == [0, 2 * N, 2 * N, 2 * N] and rows.shape == (2 * N, 0)
        assert nsp.combine(rows, order).shape == (N, 0)
        d_rows, dw = nsp.combine_backward(x, rows, order, torch.ones(N, 2).cuda())
        assert not dw.any()


def test_experts_offsets_past_32_bits(nsp):
    N, k, D = 270_000, 4, 2056  # over 2**31 elements of rows
    x = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    x[-1], x[0] = 2.0, 1.0
    ids = torch.arange(k, device="cuda").int().expand(N, k).contiguous()
    rows, order = nsp.dispatch(x, ids, k)
    assert (rows[N - 1::N] == 2).all() and (rows[::N] == 1).all()
    out = nsp.combine(rows, order)
    assert (out[-1] == 8).all() and (out[0] == 4).all() and not out[1:-1].any()
    d_rows, dw = nsp.combine_backward(x, rows, order, torch.ones(N, k, device="cuda"))
    assert torch.equal(d_rows, rows) and (dw[-1] == 4 * D).all() and not dw[1:-1].any()


def test_experts_tokens_do_not_depend_on_the_other_tokens(nsp):
    for D, dtype in ((64, "bf16"), (513, "f32"), (1001, "bf16")):
        x, ids, E, y, w, d = (t.cuda() if isinstance(t, torch.Tensor) else t
                              for t in expert_inputs(3000, 20, 4, D, dtype, D))
        _, order = nsp.dispatch(x, ids, E)
        out = nsp.combine(y, order, w)
        dw = nsp.combine_backward(d, y, order, w)[1]
        n = slice(100, 107)
        _, few = nsp.dispatch(x[n], ids[n], E)
        part = torch.zeros(7 * 4, D, dtype=y.dtype, device="cuda")
        part[few.place.view(-1).long()] = y[order.place[n].reshape(-1).long()]
        assert same(nsp.combine(part, few, w[n]), out[n])
        assert same(nsp.combine_backward(d[n], part, few, w[n])[1], dw[n])


def test_experts_gradients_and_autograd(nsp):
    x, ids, E, y, w, d = (t.cuda() if isinstance(t, torch.Tensor) else t
                          for t in expert_inputs(50, 5, 3, 24, "f32", 7))
    c = torch.randn(150, 24, generator=gen(1)).cuda()

    def value(x, w):
        rows, order = nsp.dispatch(x, ids, E)
        out = nsp.combine(torch.tanh(rows) + c, order, w)
        return (out.double() * d.double()).sum()

    leaves = [t.clone().requires_grad_() for t in (x, w)]
    grads = torch.autograd.grad(value(*leaves), leaves)
    # against PyTorch's own gradients of the formulas, in 64 bits
    _, order = nsp.dispatch(x, ids, E)
    there = ((ids >= 0) & (ids < E)).double()[..., None]
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    each = torch.tanh(xd)[:, None] + c.double()[order.place.long()]
    want = ((each * wd[..., None] * there).sum(1) * d.double()).sum()
    for a, b in zip(grads, torch.autograd.grad(want, (xd, wd))):
        assert float((a.double() - b).abs().max()) <= 1e-5 * float(b.abs().max())
    for i, t in enumerate((x, w)):  # and differences
        v = grads[i] / grads[i].abs().max()
        slope = float((grads[i].double() * v.double()).sum())
        args = [x, w]

        def f(z):
            args[i] = z
            return float(value(*args))

        assert abs(directional(f, t, v, 1e-2) - slope) <= 5e-3 * abs(slope), i
    rows, order = nsp.dispatch(leaves[0], ids, E)
    assert not any(t.requires_grad for t in order)
    (dx,) = torch.autograd.grad(rows.t().contiguous().sum() + rows[::2].sum(), leaves[0])
    dr = torch.ones(150, 24, device="cuda")
    dr[::2] += 1
    assert same(dx, nsp.dispatch_backward(dr, order))


def test_gradients_of_frozen_weights_are_not_computed(nsp, monkeypatch):
    made = {}

    def watch(name, *which):
        call = getattr(nsp._lib, name)

        def watched(*args):
            made[name] = [args[i] for i in which]
            return call(*args)

        monkeypatch.setattr(nsp._lib, name, watched)

    watch("ns_norm_backward", 6, 7)
    watch("ns_combine_backward", 9)
    x, w, b, doc, dy = (t.cuda() for t in norm_inputs(700, 520, "bf16", "f32", 4))
    full = nsp.layer_norm_backward(dy, x, w, b, *nsp.layer_norm_forward(x, w, b, doc=doc)[1:],
                                   doc=doc)
    for leaves in ((x,), (x, w), (x, b), (w,)):
        for t in (x, w, b):
            t.requires_grad_(any(t is leaf for leaf in leaves))
        y = nsp.layer_norm(x, w, b, doc=doc)
        grads = torch.autograd.grad(y, leaves, dy)
        for t, g in zip(leaves, grads):
            assert same(g, full[0 if t is x else 1 if t is w else 2])
        assert [p is not None for p in made["ns_norm_backward"]] == [
            any(t is leaf for leaf in leaves) for t in (w, b)]

    x, ids, E, _, w, d = (t.cuda() if isinstance(t, torch.Tensor) else t
                          for t in expert_inputs(300, 5, 3, 40, "bf16", 7))
    rows, order = nsp.dispatch(x, ids, E)
    full = nsp.combine_backward(d, rows, order, w)
    for leaves in ((rows,), (rows, w), (w,)):
        for t in (rows, w):
            t.requires_grad_(any(t is leaf for leaf in leaves))
        grads = torch.autograd.grad(nsp.combine(rows, order, w), leaves, d)
        for t, g in zip(leaves, grads):
            assert same(g, full[0 if t is rows else 1])
        assert (made["ns_combine_backward"][0] is not None) == (leaves[-1] is w)


# ---- all of them ---------------------------------------------------------------------------
def test_same_bits_every_time_and_on_every_stream(nsp):
    g = gen(3)
    tokens = (torch.rand(20_000, generator=g) ** 4 * 3000).int().cuda()
    dy = torch.randn(20_000, 72, generator=g).cuda()
    w = torch.randn(72, generator=g).cuda()
    ids = torch.randint(-1, 30, (20_000, 4), generator=g).int().cuda()
    gate = torch.rand(20_000, 4, generator=g).cuda()

    def once():
        y, m, r = nsp.layer_norm_forward(dy, w, w)
        rows, order = nsp.dispatch(dy, ids, 30)
        return [nsp.embed_backward(dy, tokens, 3000), y, *nsp.layer_norm_backward(dy, dy, w, w, m, r),
                rows, *order, nsp.combine(rows, order, gate),
                *nsp.combine_backward(dy, rows, order, gate)]

    first = once()
    torch.cuda.synchronize()
    again = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            again.append(once())
    torch.cuda.synchronize()
    for other in again:
        for a, b in zip(first, other):
            assert same(a, b)


@pytest.mark.parametrize("N", [100, 5000])
def test_calls_are_captured_in_a_graph(nsp, N):
    x = torch.randn(N, 80).cuda()
    w = torch.randn(80).cuda()
    table = torch.randn(500, 80).cuda()
    tokens = torch.randint(0, 500, (N,)).int().cuda()
    ids = torch.randint(-1, 9, (N, 2)).int().cuda()
    gate = torch.rand(N, 2).cuda()

    def once():
        y, m, r = nsp.layer_norm_forward(x, w, w)
        rows, order = nsp.dispatch(x, ids, 9)
        return [nsp.embed(table, tokens), nsp.embed_backward(x, tokens, 500), y,
                *nsp.layer_norm_backward(x, x, w, w, m, r), rows, *order,
                nsp.combine(rows, order, gate), *nsp.combine_backward(x, rows, order, gate),
                nsp.dispatch_backward(rows, order)]

    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        once()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:  # two of them: their workspaces are their own
        with torch.cuda.graph(graph):
            outs.append(once())
    for _ in range(2):
        x.normal_()
        table.normal_()
        tokens.random_(0, 500)
        ids.random_(-1, 9)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = once()
        for out in outs:
            for a, b in zip(out, want):
                assert same(a, b)


def refused(nsp, call):
    with pytest.raises(nsp.NsPackError) as e:
        call()
    assert e.value.code == nsp.NS_ERR_INVALID_ARG


def test_embed_refusals(nsp):
    w = torch.randn(9, 8).cuda()
    t = torch.zeros(2, 5, dtype=torch.int32).cuda()
    dy = torch.randn(2, 5, 8).cuda()
    for call in (
            lambda: nsp.embed(w.cpu(), t), lambda: nsp.embed(w, t.cpu()), lambda: nsp.embed(w, None),
            lambda: nsp.embed(w.double(), t), lambda: nsp.embed(w[0], t), lambda: nsp.embed(w.t(), t),
            lambda: nsp.embed(w, t.short()), lambda: nsp.embed(w, t.float()),
            lambda: nsp.embed(w, t.t()), lambda: nsp.embed(w, t, doc=t[:1]),
            lambda: nsp.embed(w, t, doc=t.long()), lambda: nsp.embed(w, t, scale=INF),
            lambda: nsp.embed(w, t, scale=NAN), lambda: nsp.embed(w, t, dtype=torch.float64),
            lambda: nsp.embed(w[:1].expand(9, 8), t),
            lambda: nsp.embed_backward(dy[0], t, 9), lambda: nsp.embed_backward(dy.cpu(), t, 9),
            lambda: nsp.embed_backward(dy, t, -1), lambda: nsp.embed_backward(dy, t, 2.0),
            lambda: nsp.embed_backward(dy, t, 2**32), lambda: nsp.embed_backward(dy, t, 2**31),
            lambda: nsp.embed_backward(dy.transpose(1, 2).contiguous().transpose(1, 2), t, 9),
            lambda: nsp.embed_backward(dy[:1].expand(2, 5, 8), t, 9),
            lambda: nsp.embed_backward(dy, t, 9, dtype=torch.int32),
            lambda: nsp.embed_backward(dy.double(), t, 9)):
        refused(nsp, call)


def test_layer_norm_refusals(nsp):
    x = torch.randn(4, 5, 8).cuda()
    w = torch.ones(8).cuda()
    i = torch.zeros(4, 5, dtype=torch.int32).cuda()
    y, m, r = nsp.layer_norm_forward(x, w, w)
    for call in (
            lambda: nsp.layer_norm(x.cpu()), lambda: nsp.layer_norm(x.double()),
            lambda: nsp.layer_norm(None), lambda: nsp.layer_norm(x, w[:7]),
            lambda: nsp.layer_norm(x, w.half()), lambda: nsp.layer_norm(x, w, w.half()),
            lambda: nsp.layer_norm(x, w.cpu()), lambda: nsp.layer_norm(x, w, eps=-1.0),
            lambda: nsp.layer_norm(x, w, eps=NAN), lambda: nsp.layer_norm(x, w, eps=INF),
            lambda: nsp.layer_norm(x, w, doc=i[:1]), lambda: nsp.layer_norm(x, w, doc=i.long()),
            lambda: nsp.layer_norm(x.transpose(1, 2), torch.ones(5).cuda()),
            lambda: nsp.layer_norm(x[:, :4]), lambda: nsp.layer_norm(x[..., :0]),
            lambda: nsp.layer_norm(x[0, 0, 0]), lambda: nsp.layer_norm(x[:1].expand(4, 5, 8)),
            lambda: nsp.layer_norm_backward(x[:3], x, w, w, m, r),
            lambda: nsp.layer_norm_backward(x.half(), x, w, w, m, r),
            lambda: nsp.layer_norm_backward(x, x, w, w, None, r),
            lambda: nsp.layer_norm_backward(x, x, w, w, m[:3], r),
            lambda: nsp.layer_norm_backward(x, x, w, w, m, r.half()),
            lambda: nsp.layer_norm_backward(x.transpose(1, 2), x, w, w, m, r)):
        refused(nsp, call)


def test_experts_refusals(nsp):
    x = torch.randn(6, 8).cuda()
    ids = torch.zeros(6, 2, dtype=torch.int32).cuda()
    rows, order = nsp.dispatch(x, ids, 3)
    w = torch.ones(6, 2).cuda()
    for call in (
            lambda: nsp.dispatch(x.cpu(), ids, 3), lambda: nsp.dispatch(x, ids.cpu(), 3),
            lambda: nsp.dispatch(x, ids, 0), lambda: nsp.dispatch(x, ids, 1025),
            lambda: nsp.dispatch(x, ids, 3.0), lambda: nsp.dispatch(x, ids.long(), 3),
            lambda: nsp.dispatch(x, ids[:5], 3), lambda: nsp.dispatch(x, ids[:, 0], 3),
            lambda: nsp.dispatch(x, ids[:, :0], 3), lambda: nsp.dispatch(x, ids.t().contiguous().t(), 3),
            lambda: nsp.dispatch(x[0], ids, 3), lambda: nsp.dispatch(x.t(), ids[:1].expand(8, 2), 3),
            lambda: nsp.dispatch(x.double(), ids, 3), lambda: nsp.dispatch(x, None, 3),
            lambda: nsp.combine(rows[:11], order), lambda: nsp.combine(rows, order, w[:5]),
            lambda: nsp.combine(rows, order, w.half()), lambda: nsp.combine(rows, None),
            lambda: nsp.combine(rows.double(), order), lambda: nsp.combine(rows.cpu(), order),
            lambda: nsp.combine(rows, order._replace(place=order.place.long())),
            lambda: nsp.combine(rows, order._replace(offsets=order.offsets[:1])),
            lambda: nsp.combine(rows.t().contiguous().t(), order),
            lambda: nsp.dispatch_backward(rows[:, :0].double(), order),
            lambda: nsp.combine_backward(x[:5], rows, order, w),
            lambda: nsp.combine_backward(x.half(), rows, order, w),
            lambda: nsp.combine_backward(x, rows[:11], order, w),
            lambda: nsp.combine_backward(x[:1].expand(6, 8), rows, order, w)):
        refused(nsp, call)


def test_orders_of_another_call_are_read_within_bounds(nsp):
    # places that are none of the rows', and more choices than rows: no row, no write
    rows = torch.randn(12, 8).cuda()
    place = torch.tensor([[0, 11], [12, -1], [2**31 - 1, 5], [3, -2**31], [1, 2], [40, 4]]).int().cuda()
    for last in (12, 100, -5):
        offsets = torch.tensor([0, last], dtype=torch.int32).cuda()
        order = nsp.ExpertOrder(place, place.view(-1), offsets)
        good = (place >= 0) & (place < 12)
        want = (rows[place.clamp(0, 11).long()] * good[..., None]).sum(1)
        assert torch.allclose(nsp.combine(rows, order), want, atol=1e-6)
        nsp.combine_backward(want, rows, order, torch.ones(6, 2).cuda())
    torch.cuda.synchronize()


def test_forward_mode_derivatives_are_refused(nsp):
    import torch.autograd.forward_ad as forward_ad
    x = torch.randn(6, 8).cuda()
    ids = torch.zeros(6, 2, dtype=torch.int32).cuda()
    rows, order = nsp.dispatch(x, ids, 3)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        for call in (lambda: nsp.embed(dual(x), ids), lambda: nsp.layer_norm(dual(x)),
                     lambda: nsp.layer_norm(x, dual(x[0].clone())), lambda: nsp.dispatch(dual(x), ids, 3),
                     lambda: nsp.combine(dual(rows), order),
                     lambda: nsp.combine(rows, order, dual(torch.ones(6, 2).cuda()))):
            with pytest.raises(NotImplementedError):
                call()


def test_a_model_of_them_on_a_packed_update(nsp):
    """Embedding, norms, recurrence, router, experts and loss on the packer's own arrays
    against the same formulas by PyTorch in 64 bits: loss and every gradient.  Sums of up
    to some thousand terms in 32 bits, through six layers: 2e-4 of each norm."""
    from corpus import make_preset
    c = make_preset("c1")
    pk = nsp.Packer.from_corpus(c)
    out = pk.step(0)
    tokens, pos, doc, mask = (out[n][0][:2, :256].contiguous() for n in ("tokens", "pos", "doc", "mask"))
    pk.close()
    doc[1, 200:] = -1
    B, T = tokens.shape
    V, D, E, k, K = 500, 48, 6, 2, 5
    tokens = tokens % V
    g = gen(9)

    def leaf(*shape, scale):
        return (torch.randn(*shape, generator=g) * scale).cuda()

    p = dict(table=leaf(V, D, scale=0.3), w1=1 + leaf(D, scale=0.1), b1=leaf(D, scale=0.1),
             mix=leaf(D, 2 * D, scale=0.15), w2=1 + leaf(D, scale=0.1), b2=leaf(D, scale=0.1),
             router=leaf(D, E, scale=0.4), experts=leaf(E, D, D, scale=0.15),
             head=leaf(D, V, scale=0.15))
    top, top_ids = leaf(B * T, K, scale=1.0), torch.randint(0, V, (B * T, K), generator=g).int().cuda()
    learned = (mask * (doc >= 0)).view(-1).to(torch.uint8)
    flat = doc.view(-1)

    def ours(p):
        x = nsp.embed(p["table"], tokens, scale=2.0, doc=doc)
        n = nsp.layer_norm(x, p["w1"], p["b1"], doc=doc)
        z, f = (n @ p["mix"]).chunk(2, -1)
        x = x + nsp.gated_scan(z, f, pos=pos, doc=doc)[0]
        n = nsp.layer_norm(x, p["w2"], p["b2"], doc=doc).view(B * T, D)
        r = nsp.route(n @ p["router"], k, doc=flat)
        rows, order = nsp.dispatch(n, r.ids, E)
        at = order.offsets.tolist()
        done = [torch.tanh(rows[a:b] @ w) for a, b, w in zip(at, at[1:], p["experts"])]
        x = x.view(B * T, D) + nsp.combine(torch.cat([*done, rows[at[-1]:]]), order, r.weights)
        each = nsp.distill_loss(x @ p["head"], top, top_ids, mask=learned)
        return each.sum() + 3.0 * r.loss, r.ids

    def plain(p, ids):
        real = (doc >= 0).double()[..., None]

        def norm(x, w, b):
            m = x.mean(-1, keepdim=True)
            v = ((x - m) ** 2).mean(-1, keepdim=True)
            return ((x - m) / torch.sqrt(v + 1e-5) * w + b) * real

        x = p["table"][tokens.long()] * 2.0 * real
        z, f = (norm(x, p["w1"], p["b1"]) @ p["mix"]).chunk(2, -1)
        a = torch.sigmoid(f)
        h, ys = torch.zeros(B, D, dtype=torch.float64, device="cuda"), []
        for t in range(T):
            prev = h * (pos[:, t] != 0).double()[:, None]
            new = a[:, t] * prev + (1 - a[:, t]) * z[:, t]
            h = torch.where(real[:, t] > 0, new, h)
            ys.append(new * real[:, t])
        x = x + torch.stack(ys, 1)
        n = norm(x, p["w2"], p["b2"]).view(B * T, D)
        probs = torch.softmax(n @ p["router"], -1)
        there = (ids >= 0).double()
        chosen = probs.gather(1, ids.clamp(min=0).long()) * there
        w = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
        every = torch.tanh(torch.einsum("nd,edf->nef", n, p["experts"]))
        each = every.gather(1, ids.clamp(min=0).long()[..., None].expand(-1, -1, D))
        x = x.view(B * T, D) + (each * (w * there)[..., None]).sum(1)
        log_q = torch.log_softmax(x @ p["head"], -1).gather(1, top_ids.long())
        pt = torch.softmax(top.double(), -1)
        loss = ((pt * (pt.log() - log_q)).sum(1) * learned.double()).sum()
        M = float((flat >= 0).sum())
        counts = torch.stack([(ids == e).sum() for e in range(E)]).double()
        balance = E / (k * M * M) * (counts * (probs * real.view(-1, 1)).sum(0)).sum()
        return loss + 3.0 * balance

    mine = {n: t.clone().requires_grad_() for n, t in p.items()}
    loss, ids = ours(mine)
    got = dict(zip(mine, torch.autograd.grad(loss, list(mine.values()))))
    exact = {n: t.double().requires_grad_() for n, t in p.items()}
    value = plain(exact, ids)
    want = dict(zip(exact, torch.autograd.grad(value, list(exact.values()))))
    assert abs(float(loss.detach()) - float(value.detach())) <= 2e-5 * abs(float(value.detach()))
    for n in p:
        assert float((got[n].double() - want[n]).norm()) <= 2e-4 * float(want[n].norm()), n


def test_readme_lines_run_on_an_update(nsp):
    import os
    from corpus import make_preset
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    lines = text.split("### Training on the packed rows")[1].split("```python\n")[2].split("```")[0]
    c = make_preset("c1")
    pk = nsp.Packer.from_corpus(c)
    out = pk.step(0)
    pk.close()
    v = {n: out[n][0] for n in ("tokens", "doc")}
    flat = v["doc"].view(-1)
    v.update(table=torch.randn(c.vocab, 32).cuda(), gain=torch.ones(32).cuda(),
             shift=torch.zeros(32).cuda(),
             r=nsp.route(torch.randn(flat.numel(), 16).cuda(), 2, doc=flat))
    exec(lines, v)
    want = (v["r"].weights * (1 + (v["r"].ids == 3))).sum(1, keepdim=True) * v["x"]
    assert torch.allclose(v["out"], want, atol=1e-5) and not v["out"][flat < 0].any()

"""More operators of a model trained on packed rows: cases, inputs, plain forms.

What stands around the recurrence, the router and the loss in such a model:

* ``embed`` / ``embed_backward``: the rows of a table at a batch's tokens, scaled,
  and the table's gradient; padding (``doc < 0``) has rows of 0 and no gradient;
* ``layer_norm`` and its passes: the norm of every real position, its gradient and
  those of the weight and the bias;
* ``dispatch`` / ``combine`` and their backward passes: tokens sorted by the experts
  that a router chose (-1: none), and the experts' rows brought back, times the
  router's weights.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the framework's operators.  ``exact`` computes it from
the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _nsp():
    import deterministic_packed_assembly_gb300 as nsp
    return nsp


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # the tokens that 64 sequences have just generated
        dict(name="embed_one_token", op="embed", B=64, T=1, V=32000, D=2048, dtype="bf16",
             wtype="bf16", train=False, packed=False, skew=True, scaled=False, wide_ids=True),
        # the forward pass of a small model on one update of 16 rows of 1024 (validation),
        # 32-bit weights and 16-bit activations
        dict(name="embed_forward", op="embed", B=16, T=1024, V=32000, D=1280, dtype="bf16",
             wtype="f32", train=False, packed=True, skew=True, scaled=True, wide_ids=False),
        # a training step on 8 packed rows of 4096, a large vocabulary: most rows of the
        # gradient are 0, a few tokens make up much of the batch
        dict(name="embed_train", op="embed", B=8, T=4096, V=128256, D=2560, dtype="bf16",
             wtype="bf16", train=True, packed=True, skew=True, scaled=False, wide_ids=False),
        # one odd batch of tokens drawn evenly, odd vocabulary and width, 32 bits
        dict(name="embed_train_odd", op="embed", B=1, T=99991, V=50257, D=1001, dtype="f32",
             wtype="f32", train=True, packed=True, skew=False, scaled=True, wide_ids=False),
        # the norm of one generated token for each of 64 sequences
        dict(name="norm_one_token", op="norm", B=64, T=1, D=2048, dtype="bf16", wtype="bf16",
             train=False, packed=False, bias=True),
        # a training step's norm on 8 packed rows of 4096, 32-bit weights
        dict(name="norm_train", op="norm", B=8, T=4096, D=2560, dtype="bf16", wtype="f32",
             train=True, packed=True, bias=True),
        # odd numbers of rows and channels, 32-bit activations
        dict(name="norm_train_odd", op="norm", B=1, T=9973, D=5003, dtype="f32", wtype="f32",
             train=True, packed=True, bias=True),
        # few wide rows, no bias (a large model's validation)
        dict(name="norm_forward_wide", op="norm", B=3, T=1361, D=16384, dtype="f16", wtype="f16",
             train=False, packed=True, bias=False),
        # the experts of one generated token for each of 64 sequences
        dict(name="experts_one_token", op="experts", N=64, E=64, k=8, D=2048, dtype="bf16",
             train=False, pad=0.0),
        # a training step's tokens on 8 rows of 4096, 64 experts
        dict(name="experts_train", op="experts", N=32768, E=64, k=8, D=2560, dtype="bf16",
             train=True, pad=0.03),
        # odd numbers of tokens, experts and channels, two experts a token
        dict(name="experts_train_odd", op="experts", N=9973, E=60, k=2, D=1001, dtype="f32",
             train=True, pad=0.1),
        # many tokens of many experts, narrow rows: the sort's share is the largest
        dict(name="experts_forward_many", op="experts", N=131072, E=256, k=8, D=512, dtype="bf16",
             train=False, pad=0.03),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "experts"])
    train = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "experts":
        E = rng.choice([8, 16, 60, 64, 128, 256, _log(rng, 4, 512)])
        c = dict(op=op, N=_log(rng, 16, 131072), E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])),
                 D=_log(rng, 64, 4096), dtype=dtype, train=train, pad=rng.choice([0.0, 0.03, 0.2]))
        rows, most = "N", work(listed()[9])["bytes"]
    else:
        T = 1 if rng.random() < 0.2 else _log(rng, 2, 32768)
        B = _log(rng, 1, 64 if T > 1 else 256)
        packed = T > 1 and rng.random() < 0.8
        c = dict(op=op, B=B, T=T, dtype=dtype, wtype=rng.choice([dtype, dtype, "f32"]),
                 train=train, packed=packed)
        if op == "embed":
            V = rng.choice([32000, 50257, 64000, 128256, 151936, _log(rng, 1000, 151936)])
            D = _log(rng, 64, 4096)
            c.update(V=V, D=max(64, min(D, (128256 * 2560 * 2) // (V * BYTES[c["wtype"]]))),
                     skew=rng.random() < 0.7, scaled=rng.random() < 0.5,
                     wide_ids=rng.random() < 0.3)
            rows, most = "B", 2 * 128256 * 2560 * 2
        else:
            c.update(D=_log(rng, 64, 16384), bias=rng.random() < 0.7)
            rows, most = "B", work(listed()[5])["bytes"]
    while work(c)["bytes"] > most and c[rows] > 1:
        c[rows] = max(1, c[rows] * 2 // 3)
    while work(c)["bytes"] > most:
        c["T"] = c["T"] * 2 // 3
    return c


# ---- inputs --------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _packed_rows(g, B, T, median=400.0):
    """Document ids of packed rows: log-normal lengths, a padded end on most rows."""
    start = torch.rand((B, T), generator=g, device=DEV) < 1.0 / (1.6 * median)
    start[:, 0] = True
    t = torch.arange(T, device=DEV).expand(B, T)
    doc = start.int().cumsum(1) - 1
    pad = (torch.rand((B, 1), generator=g, device=DEV) * 0.04 * T).long()
    return torch.where(t >= T - pad, torch.full_like(doc, -1), doc).int().contiguous()


def _shares(V, skew):
    """How often each token comes: as 1 / rank, the frequent ones first, or evenly."""
    if not skew:
        return torch.full((V,), 1.0 / V, dtype=torch.float64)
    p = 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)
    return p / p.sum()


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, device=DEV).normal_(mean, scale, generator=g).to(dtype)

    if case["op"] == "embed":
        B, T, V, D = case["B"], case["T"], case["V"], case["D"]
        s["weight"] = normal(V, D, scale=0.02, dtype=DTYPES[case["wtype"]])
        border = _shares(V, case["skew"]).cumsum(0).to(DEV)
        u = torch.rand((B, T), generator=g, device=DEV, dtype=torch.float64)
        tokens = torch.searchsorted(border, u).clamp(max=V - 1)
        s["doc"] = _packed_rows(g, B, T) if case["packed"] else None
        if case["packed"]:
            tokens = torch.where(s["doc"] >= 0, tokens, torch.zeros_like(tokens))
        s["tokens"] = tokens if case["wide_ids"] else tokens.int()
        s["scale"] = math.sqrt(D) if case["scaled"] else 1.0
        if case["train"]:
            s["dy"] = normal(B, T, D, scale=1e-2, dtype=dt)
    elif case["op"] == "norm":
        B, T, D = case["B"], case["T"], case["D"]
        # a residual stream: rows of several sizes, a mean, a few channels that stand out
        size = torch.empty((B, T, 1), device=DEV).uniform_(0.5, 8.0, generator=g)
        x = normal(B, T, D, mean=0.1) * size
        x[..., ::997] *= 20.0
        s["x"] = x.to(dt)
        s["weight"] = normal(D, scale=0.2, mean=1.0, dtype=DTYPES[case["wtype"]])
        s["bias"] = normal(D, scale=0.1, dtype=DTYPES[case["wtype"]]) if case["bias"] else None
        s["eps"] = 1e-5
        s["doc"] = _packed_rows(g, B, T) if case["packed"] else None
        if case["train"]:
            s["dy"] = normal(B, T, D, scale=1e-2, dtype=dt)
    else:
        N, E, k, D = case["N"], case["E"], case["k"], case["D"]
        s["x"] = normal(N, D, dtype=dt)
        # a router's choice: some experts are chosen more often than others
        top, ids = (normal(N, E) + normal(1, E, scale=0.7)).topk(k, dim=1)
        w = torch.softmax(top, 1)
        if case["pad"]:
            gone = torch.rand((N + 63) // 64, generator=g, device=DEV) < case["pad"]
            gone = gone.repeat_interleave(64)[:N, None]
            ids, w = ids.masked_fill(gone, -1), w.masked_fill(gone, 0.0)
        s["ids"], s["weights"] = ids.int().contiguous(), w.contiguous()
        s["expert_rows"] = normal(N * k, D, dtype=dt)  # what the experts computed, in their order
        if case["train"]:
            s["d_out"] = normal(N, D, scale=1e-2, dtype=dt)
            s["d_rows"] = normal(N * k, D, scale=1e-2, dtype=dt)
    return s


# ---- plain forms ----------------------------------------------------------------
def _plain_embed(s):
    c = s["case"]
    ids = s["tokens"].long()
    y = s["weight"][ids].float() * s["scale"]
    if s["doc"] is not None:
        y = torch.where((s["doc"] >= 0)[..., None], y, torch.zeros_like(y))
    out = dict(y=y.to(DTYPES[c["dtype"]]))
    if c["train"]:
        dy = s["dy"].float() * s["scale"]
        if s["doc"] is not None:
            dy = torch.where((s["doc"] >= 0)[..., None], dy, torch.zeros_like(dy))
        d = torch.zeros((c["V"], c["D"]), device=DEV)
        d.index_add_(0, ids.reshape(-1), dy.reshape(-1, c["D"]))
        out["dweight"] = d.to(s["weight"].dtype)
    return out


def _plain_norm(s):
    c = s["case"]
    x, w = s["x"].float(), s["weight"].float()
    real = None if s["doc"] is None else (s["doc"] >= 0)[..., None]
    d = x - x.mean(-1, keepdim=True)
    rstd = ((d * d).mean(-1, keepdim=True) + s["eps"]).rsqrt()
    xh = d * rstd
    y = xh * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if real is not None:
        y = torch.where(real, y, torch.zeros_like(y))
    out = dict(y=y.to(s["x"].dtype))
    if not c["train"]:
        return out
    dy = s["dy"].float()
    if real is not None:
        dy = torch.where(real, dy, torch.zeros_like(dy))
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    out["dx"] = dx.to(s["x"].dtype)
    out["dweight"] = (dy * xh).sum((0, 1)).to(s["weight"].dtype)
    if s["bias"] is not None:
        out["dbias"] = dy.sum((0, 1)).to(s["bias"].dtype)
    return out


def _plain_experts(s):
    c = s["case"]
    N, E, k, D = c["N"], c["E"], c["k"], c["D"]
    ids = s["ids"].reshape(-1).long()
    key = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E))
    slots = torch.sort(key, stable=True).indices
    place = torch.empty_like(slots)
    place[slots] = torch.arange(N * k, device=DEV)
    counts = torch.zeros(E + 1, dtype=torch.long, device=DEV)
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:E].cumsum(0)])
    token = slots // k
    there = (key[slots] < E)[:, None]
    rows = s["x"][token]
    rows = torch.where(there, rows, torch.zeros_like(rows))
    place = place.view(N, k)
    chosen = (key.view(N, k) < E)[..., None]
    w = s["weights"][..., None]
    each = s["expert_rows"][place].float()
    each = torch.where(chosen, each, torch.zeros_like(each))
    out = dict(rows=rows, place=place.int(), slots=slots.int(), offsets=offsets.int(),
               out=(each * w).sum(1).to(s["x"].dtype))
    if not c["train"]:
        return out
    d = s["d_out"].float()
    out["d_weights"] = (each * d[:, None]).sum(2)
    d_rows = d[token] * s["weights"].reshape(-1)[slots][:, None]
    out["d_expert_rows"] = torch.where(there, d_rows, torch.zeros_like(d_rows)).to(s["x"].dtype)
    each = s["d_rows"][place].float()
    out["dx"] = torch.where(chosen, each, torch.zeros_like(each)).sum(1).to(s["x"].dtype)
    return out


# ---- one pass ---------------------------------------------------------------------
def _own_embed(s):
    nsp = _nsp()
    c = s["case"]
    out = dict(y=nsp.embed(s["weight"], s["tokens"], scale=s["scale"], doc=s["doc"],
                           dtype=DTYPES[c["dtype"]]))
    if c["train"]:
        out["dweight"] = nsp.embed_backward(s["dy"], s["tokens"], c["V"], scale=s["scale"],
                                            doc=s["doc"], dtype=s["weight"].dtype)
    return out


def _own_norm(s):
    nsp = _nsp()
    if not s["case"]["train"]:
        return dict(y=nsp.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], doc=s["doc"]))
    y, mean, rstd = nsp.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=s["eps"],
                                           doc=s["doc"])
    dx, dweight, dbias = nsp.layer_norm_backward(s["dy"], s["x"], s["weight"], s["bias"], mean,
                                                 rstd, doc=s["doc"])
    out = dict(y=y, dx=dx, dweight=dweight)
    if s["bias"] is not None:
        out["dbias"] = dbias
    return out


def _own_experts(s):
    nsp = _nsp()
    c = s["case"]
    rows, order = nsp.dispatch(s["x"], s["ids"], c["E"])
    out = dict(rows=rows, place=order.place, slots=order.slots, offsets=order.offsets,
               out=nsp.combine(s["expert_rows"], order, s["weights"]))
    if c["train"]:
        out["d_expert_rows"], out["d_weights"] = nsp.combine_backward(
            s["d_out"], s["expert_rows"], order, s["weights"])
        out["dx"] = nsp.dispatch_backward(s["d_rows"], order)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(embed=_own_embed, norm=_own_norm, experts=_own_experts)[op](state)
    return dict(embed=_plain_embed, norm=_plain_norm, experts=_plain_experts)[op](state)


# ---- what one pass cannot do without -------------------------------------------------
def work(case):
    es, D = BYTES[case["dtype"]], case["D"]
    if case["op"] == "embed":
        N, V, ws = case["B"] * case["T"], case["V"], BYTES[case["wtype"]]
        # rows of the table that are there at all among N tokens, on average
        used = float((1.0 - (N * torch.log1p(-_shares(V, case["skew"]))).exp()).sum())
        moved = used * D * ws + N * D * es + N * (8 if case["wide_ids"] else 4)
        moved += 4 * N if case["packed"] else 0
        if case["train"]:  # dy in, the table's gradient out
            moved += N * D * es + V * D * ws
        return dict(bytes=moved, flops=N * D * (3 if case["train"] else 1))
    if case["op"] == "norm":
        N, ws = case["B"] * case["T"], BYTES[case["wtype"]]
        vectors = (2 if case["bias"] else 1) * D * ws
        moved = 2 * N * D * es + vectors + (4 * N if case["packed"] else 0)
        if case["train"]:  # dy in, x again, dx and the weights' gradients out
            moved += 3 * N * D * es + vectors
        return dict(bytes=moved, flops=N * D * (22 if case["train"] else 8))
    N, k = case["N"], case["k"]
    S = N * k
    there = (1.0 - case["pad"]) * S
    moved = N * D * es + S * D * es + 12 * S + 4 * case["E"]  # dispatch
    moved += there * D * es + N * D * es + 4 * S              # combine
    if case["train"]:
        moved += N * D * es + there * D * es + S * D * es + 4 * S  # d_out, rows in; d_rows, d_weights
        moved += there * D * es + N * D * es                       # d_rows in, dx
    return dict(bytes=moved, flops=there * D * (6 if case["train"] else 2))


# ---- the definitions, in 64 bits --------------------------------------------------------
def _exact_embed(case, s):
    real = torch.ones(s["tokens"].shape, device=DEV, dtype=torch.float64)
    if s["doc"] is not None:
        real = (s["doc"] >= 0).double()
    flat = s["tokens"].reshape(-1).long()
    y = s["weight"].double().index_select(0, flat).view(*s["tokens"].shape, case["D"])
    out = dict(y=y.mul_(real[..., None] * s["scale"]))
    if case["train"]:  # each token's gradients one after the other, tokens side by side
        dweight = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device=DEV)
        keep = torch.nonzero(real.reshape(-1))[:, 0]
        order = keep[torch.argsort(flat[keep], stable=True)]
        dy = s["dy"].reshape(-1, case["D"])
        # the n-th position of every token at a time, the frequent ones' many by sums
        ids, counts = torch.unique_consecutive(flat[order], return_counts=True)
        first = counts.cumsum(0) - counts
        n = 0
        while n < 64 and bool((counts > n).any()):
            some = counts > n
            dweight[ids[some]] += dy[order[first[some] + n]].double() * s["scale"]
            n += 1
        for i in torch.nonzero(counts > n)[:, 0].tolist():
            a, b = int(first[i]) + n, int(first[i] + counts[i])
            dweight[ids[i]] += dy[order[a:b]].double().sum(0) * s["scale"]
        out["dweight"] = dweight
    return out


def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    b = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
    gone = torch.zeros(x.shape[:2], dtype=torch.bool, device=DEV)
    if s["doc"] is not None:
        gone = s["doc"] < 0
    D = case["D"]
    mean = x.sum(-1, keepdim=True) / D
    sigma = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / D + s["eps"])
    out = dict(y=((x - mean) / sigma * w + b).masked_fill(gone[..., None], 0.0))
    if not case["train"]:
        return out
    dy = s["dy"].double().masked_fill(gone[..., None], 0.0)
    unit = (x - mean) / sigma
    d_unit = dy * w
    # through the deviation, then through the mean
    d_dev = d_unit / sigma - unit * (d_unit * unit).sum(-1, keepdim=True) / (D * sigma)
    out["dx"] = d_dev - d_dev.sum(-1, keepdim=True) / D
    out["dweight"] = torch.einsum("btd,btd->d", dy, unit)
    if s["bias"] is not None:
        out["dbias"] = torch.einsum("btd->d", dy)
    return out


def _exact_experts(case, s):
    N, E, k, D = case["N"], case["E"], case["k"], case["D"]
    ids = s["ids"].reshape(-1)
    groups = [torch.nonzero(ids == e)[:, 0] for e in range(E)]  # each expert's slots, in order
    there = torch.cat(groups)
    slots = torch.cat([there, torch.nonzero((ids < 0) | (ids >= E))[:, 0]])
    place = torch.argsort(slots).view(N, k)
    offsets = torch.tensor([0] + [len(g) for g in groups]).cumsum(0)
    M = len(there)

    def blank(*shape):
        return torch.zeros(shape, dtype=torch.float64, device=DEV)

    out = dict(place=place.int(), slots=slots.int(), offsets=offsets.int(), rows=blank(N * k, D),
               out=blank(N, D))
    if case["train"]:
        out.update(d_weights=blank(N, k), d_expert_rows=blank(N * k, D), dx=blank(N, D))
    out["rows"][:M] = s["x"][there // k].double()
    for j in range(k):  # the tokens' j-th choices
        n = torch.nonzero(place[:, j] < M)[:, 0]
        at, w = place[n, j], s["weights"][n, j].double()[:, None]
        y = s["expert_rows"][at].double()
        out["out"][n] += w * y
        if case["train"]:
            d = s["d_out"][n].double()
            out["d_weights"][n, j] = torch.einsum("nd,nd->n", d, y)
            out["d_expert_rows"][at] = w * d
            out["dx"][n] += s["d_rows"][at].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(embed=_exact_embed, norm=_exact_norm, experts=_exact_experts)[case["op"]](case, s)

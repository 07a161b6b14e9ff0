"""Operators of a model trained on packed rows: cases, inputs, plain forms.

Three operators take a packed batch's position ids, document ids and loss mask
next to a model's activations:

* ``gated_scan``: the gated linear recurrence over time that starts again at
  every document (``pos == 0``) and passes over padding (``doc < 0``);
* ``distill_loss``: the divergence from a teacher's top logits, on the learned
  positions only;
* ``route``: a router's choice of experts, its per-expert counts and its balance
  loss, over the real positions only.

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
NEG_INF = float("-inf")


def _nsp():
    import deterministic_packed_assembly_gb300 as nsp
    return nsp


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # one token for each of 64 sequences being generated: state in, state out
        dict(name="scan_one_token", op="scan", B=64, T=1, D=2048, dtype="bf16", train=False,
             state=True, packed=False, joint=False),
        # the forward pass of a small model on one update of 16 rows of 1024
        # (validation); z and f are the halves of one projection
        dict(name="scan_forward", op="scan", B=16, T=1024, D=1280, dtype="bf16", train=False,
             state=False, packed=True, joint=True),
        # a training step's layer on 8 packed rows of 4096
        dict(name="scan_train", op="scan", B=8, T=4096, D=2560, dtype="bf16", train=True,
             state=False, packed=True, joint=True),
        # one long row, odd length and width, 32-bit activations, state carried in
        # (a long context continued from the previous chunk)
        dict(name="scan_train_long", op="scan", B=1, T=32749, D=1001, dtype="f32", train=True,
             state=True, packed=True, joint=False),
        # evaluation of a few rows: latency
        dict(name="distill_small", op="distill", N=64, V=32000, K=16, dtype="bf16",
             tdtype="f32", train=False, temperature=1.0, tail=False, learned=1.0),
        # evaluation loss over validation rows, odd vocabulary
        dict(name="distill_eval", op="distill", N=4093, V=50257, K=32, dtype="bf16",
             tdtype="bf16", train=False, temperature=1.0, tail=True, learned=0.95),
        # supervised fine-tuning rows, completion tokens learned only: loss and
        # gradient of the logits
        dict(name="distill_train", op="distill", N=8192, V=128256, K=64, dtype="bf16",
             tdtype="bf16", train=True, temperature=1.0, tail=False, learned=0.65),
        # 32-bit logits, odd vocabulary, softened teacher whose tail is left out
        dict(name="distill_train_soft", op="distill", N=1021, V=50257, K=200, dtype="f32",
             tdtype="f32", train=True, temperature=2.0, tail=True, learned=0.9),
        # the router of one generated token for each of 64 sequences
        dict(name="route_one_token", op="route", N=64, E=64, k=8, dtype="f32", train=False,
             normalize=True, pad=0.0),
        # a training step's router on 8 rows of 4096, 64 experts
        dict(name="route_train", op="route", N=32768, E=64, k=8, dtype="f32", train=True,
             normalize=True, pad=0.03),
        # a large global batch, 256 experts, 16-bit logits (ties are frequent)
        dict(name="route_train_wide", op="route", N=262144, E=256, k=8, dtype="bf16",
             train=True, normalize=False, pad=0.03),
        # odd numbers of tokens and experts, two experts a token
        dict(name="route_odd", op="route", N=99991, E=60, k=2, dtype="bf16", train=True,
             normalize=True, pad=0.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["scan", "distill", "route"])
    train = rng.random() < 0.6
    if op == "scan":
        T = 1 if rng.random() < 0.2 else _log(rng, 2, 32768)
        D = _log(rng, 64, 2560)
        B = _log(rng, 1, 64 if T > 1 else 256)
        B = max(1, min(B, 8 * 4096 * 2560 // (T * D)))
        return dict(op=op, B=B, T=T, D=D, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    train=train, state=T == 1 or rng.random() < 0.4,
                    packed=T > 1 and rng.random() < 0.8, joint=rng.random() < 0.5)
    if op == "distill":
        V = rng.choice([32000, 50257, 64000, 128256, 151936, _log(rng, 1000, 151936)])
        N = max(1, min(_log(rng, 16, 16384), 6000 * 128256 // V))
        soft = rng.random() < 0.4
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            N = max(1, N // 2)
        return dict(op=op, N=N, V=V, K=min(V, _log(rng, 1, 256)), dtype=dtype,
                    tdtype=rng.choice(["bf16", "f32"]), train=train,
                    temperature=rng.choice([1.5, 2.0, 4.0]) if soft else 1.0,
                    tail=rng.random() < 0.5, learned=rng.choice([1.0, 0.95, 0.65]))
    E = rng.choice([8, 16, 64, 128, 256, _log(rng, 4, 512)])
    N = max(1, min(_log(rng, 16, 524288), 262144 * 256 // E))
    return dict(op=op, N=N, E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])),
                dtype=rng.choice(["f32", "f32", "bf16"]), train=train,
                normalize=rng.random() < 0.6, pad=rng.choice([0.0, 0.03, 0.2]))


# ---- inputs --------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _packed_rows(g, B, T, median=400.0):
    """Position and document ids of packed rows: log-normal document lengths, a
    padded end on most rows."""
    start = torch.rand((B, T), generator=g, device=DEV) < 1.0 / (1.6 * median)
    start[:, 0] = True
    t = torch.arange(T, device=DEV).expand(B, T)
    pos = t - torch.where(start, t, torch.zeros_like(t)).cummax(1).values
    doc = start.int().cumsum(1) - 1
    pad = (torch.rand((B, 1), generator=g, device=DEV) * 0.04 * T).long()
    padded = t >= T - pad
    return (torch.where(padded, torch.zeros_like(pos), pos).int().contiguous(),
            torch.where(padded, torch.full_like(doc, -1), doc).int().contiguous())


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, device=DEV).normal_(mean, scale, generator=g).to(dtype)

    if case["op"] == "scan":
        B, T, D = case["B"], case["T"], case["D"]
        if case["joint"]:
            both = normal(B, T, 2 * D, dtype=dt)
            s["z"], s["f"] = both[..., :D], both[..., D:]
        else:
            s["z"], s["f"] = normal(B, T, D, dtype=dt), normal(B, T, D, dtype=dt)
        # forget-gate biases from short memories to long ones
        s["bias"] = torch.empty(D, device=DEV).uniform_(0.0, 6.0, generator=g)
        s["pos"], s["doc"] = _packed_rows(g, B, T) if case["packed"] else (None, None)
        if case["packed"] and case["state"]:
            s["pos"][0, :] += torch.where(s["doc"][0] == 0, 4096, 0).int()  # goes on from before
        s["h0"] = normal(B, D) if case["state"] else None
        if case["train"]:
            s["dy"] = normal(B, T, D, scale=1e-2, dtype=dt)
            s["dh"] = normal(B, D, scale=1e-2) if case["state"] else None
    elif case["op"] == "distill":
        N, V, K = case["N"], case["V"], case["K"]
        logits = torch.empty((N, V), device=DEV, dtype=dt)
        top_ids = torch.empty((N, K), device=DEV, dtype=torch.int32)
        top = torch.empty((N, K), device=DEV, dtype=DTYPES[case["tdtype"]])
        rows = max(1, (1 << 28) // V)
        for a in range(0, N, rows):  # a teacher that agrees with the student in part
            x = normal(min(rows, N - a), V, scale=2.5)
            logits[a:a + rows] = x
            v, i = (x + normal(*x.shape, scale=1.2)).topk(K, dim=1)
            top[a:a + rows], top_ids[a:a + rows] = v, i
        s.update(logits=logits, top=top, top_ids=top_ids, temperature=case["temperature"])
        s["lse"] = None
        if case["tail"]:  # the teacher's top logits hold 70 to 99 % of its probability
            share = torch.empty(N, device=DEV).uniform_(0.70, 0.99, generator=g)
            s["lse"] = (top.float() / case["temperature"]).logsumexp(1) - share.log()
        s["mask"] = None
        if case["learned"] < 1.0:  # prompts of a fixed share of every document
            pos, doc = _packed_rows(g, 1, N, 200.0)
            length = torch.bincount(doc[0].clamp(min=0).long(), minlength=1)
            s["mask"] = ((pos[0] >= (1.0 - case["learned"]) * length[doc[0].clamp(min=0).long()])
                         & (doc[0] >= 0)).to(torch.uint8)
        if case["train"]:  # the update's loss is the mean over its learned positions
            learned = N if s["mask"] is None else int(s["mask"].sum())
            s["weight"] = torch.full((N,), 1.0 / max(1, learned), device=DEV)
    else:
        N, E, k = case["N"], case["E"], case["k"]
        s["logits"] = (normal(N, E) + normal(1, E, scale=0.7)).to(dt)
        s["doc"] = None
        if case["pad"]:
            doc = torch.arange(N, device=DEV, dtype=torch.int32) // 400
            gone = torch.rand((N + 63) // 64, generator=g, device=DEV) < case["pad"]
            s["doc"] = torch.where(gone.repeat_interleave(64)[:N], torch.full_like(doc, -1), doc)
        if case["train"]:
            s["d_weights"] = normal(N, k, scale=1e-2)
            s["d_loss"] = torch.full((), 1e-2, device=DEV)
    return s


# ---- plain forms ----------------------------------------------------------------
def _scan_doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, h_{-1} = 0, by doubling."""
    T, step = a.shape[1], 1
    while step < T:
        b = torch.cat([b[:, :step], torch.addcmul(b[:, step:], a[:, step:], b[:, :-step])], 1)
        if 2 * step < T:
            a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    z, x = s["z"].float(), s["f"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    a, keep = torch.sigmoid(x), torch.sigmoid(-x)
    real = None if s["doc"] is None else (s["doc"] >= 0)[..., None]
    carry = a
    if s["pos"] is not None:
        carry = torch.where((s["pos"] == 0)[..., None], torch.zeros_like(a), a)
    b = keep * z
    if real is not None:
        carry = torch.where(real, carry, torch.ones_like(a))
        b = torch.where(real, b, torch.zeros_like(b))
    first = b[:, :1] if s["h0"] is None else b[:, :1] + carry[:, :1] * s["h0"][:, None]
    h = _scan_doubling(carry, torch.cat([first, b[:, 1:]], 1))
    y = h if real is None else torch.where(real, h, torch.zeros_like(h))
    out = dict(y=y.to(s["z"].dtype), h_last=h[:, -1].clone())
    if not c["train"]:
        return out
    dy = s["dy"].float()
    if real is not None:
        dy = torch.where(real, dy, torch.zeros_like(dy))
    last = dy[:, -1:] if s["dh"] is None else dy[:, -1:] + s["dh"][:, None]
    following = torch.cat([carry[:, 1:], torch.ones_like(carry[:, :1])], 1)
    d = _scan_doubling(following.flip(1), torch.cat([dy[:, :-1], last], 1).flip(1)).flip(1)
    zero = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([zero, h[:, :-1]], 1)
    if s["pos"] is not None:
        before = torch.where((s["pos"] == 0)[..., None], torch.zeros_like(before), before)
    dz, df = d * keep, a * keep * d * (before - z)
    if real is not None:
        dz, df = (torch.where(real, v, torch.zeros_like(v)) for v in (dz, df))
    out.update(dz=dz.to(s["z"].dtype), df=df.to(s["f"].dtype), dbias=df.sum((0, 1)))
    if s["h0"] is not None:
        out["dh0"] = (carry[:, :1] * d[:, :1])[:, 0].clone()
    return out


def _plain_distill(s):
    tau = 1.0 / s["temperature"]
    x = s["logits"].float() * tau
    lse = torch.logsumexp(x, 1)
    t = s["top"].float() * tau
    ids = s["top_ids"].long()
    log_p = t - (torch.logsumexp(t, 1) if s["lse"] is None else s["lse"])[:, None]
    p = log_p.exp()
    loss = (p * (log_p - (x.gather(1, ids) - lse[:, None]))).sum(1) * s["temperature"] ** 2
    if s["mask"] is not None:
        loss = torch.where(s["mask"] != 0, loss, torch.zeros_like(loss))
    if not s["case"]["train"]:
        return dict(loss=loss)
    g = x.sub_(lse[:, None]).exp_()
    if s["lse"] is not None:
        g *= p.sum(1, keepdim=True)
    g.scatter_add_(1, ids, -p)
    w = s["weight"] * s["temperature"]
    g *= w[:, None]
    if s["mask"] is not None:
        g = torch.where((s["mask"] != 0)[:, None], g, torch.zeros_like(g))
    return dict(loss=loss, dlogits=g.to(s["logits"].dtype))


def _plain_route(s):
    c = s["case"]
    N, E, k = c["N"], c["E"], c["k"]
    x = s["logits"].float()
    real = torch.ones(N, dtype=torch.bool, device=DEV) if s["doc"] is None else s["doc"] >= 0
    e = (x - x.amax(1, keepdim=True)).exp()
    p = e / e.sum(1, keepdim=True)
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = p.gather(1, ids)
    total = chosen.sum(1, keepdim=True)
    w = chosen / total if c["normalize"] else chosen
    w = torch.where(real[:, None], w, torch.zeros_like(w))
    one = torch.zeros((N, E), device=DEV).scatter_(1, ids, real[:, None].float().expand(N, k))
    counts = one.sum(0)
    tokens = real.sum()
    mass = torch.where(real[:, None], p, torch.zeros_like(p)).sum(0)
    coef = E / (k * tokens.float().clamp(min=1) ** 2)
    loss = coef * (counts * mass).sum()
    out = dict(ids=torch.where(real[:, None], ids, torch.full_like(ids, -1)).int(), weights=w,
               counts=counts.int(), tokens=tokens.int(), loss=loss)
    if not c["train"]:
        return out
    g = (s["d_loss"] * coef * counts).expand(N, E)
    if c["normalize"]:
        dchosen = (s["d_weights"] - (w * s["d_weights"]).sum(1, keepdim=True)) / total
    else:
        dchosen = s["d_weights"]
    g = g.scatter_add(1, ids, dchosen)
    d = p * (g - (p * g).sum(1, keepdim=True))
    out["dlogits"] = torch.where(real[:, None], d, torch.zeros_like(d)).to(s["logits"].dtype)
    return out


# ---- one pass ---------------------------------------------------------------------
def _own_scan(s):
    nsp = _nsp()
    if not s["case"]["train"]:
        y, h = nsp.gated_scan(s["z"], s["f"], s["bias"], pos=s["pos"], doc=s["doc"], h0=s["h0"])
        return dict(y=y, h_last=h)
    y, h, carry = nsp.gated_scan_forward(s["z"], s["f"], s["bias"], pos=s["pos"], doc=s["doc"],
                                         h0=s["h0"])
    dz, df, dbias, dh0 = nsp.gated_scan_backward(s["dy"], s["dh"], s["z"], s["f"], s["bias"], carry,
                                                 pos=s["pos"], doc=s["doc"])
    out = dict(y=y, h_last=h, dz=dz, df=df, dbias=dbias)
    if s["h0"] is not None:
        out["dh0"] = dh0
    return out


def _own_distill(s):
    nsp = _nsp()
    kw = dict(mask=s["mask"], temperature=s["temperature"], teacher_lse=s["lse"])
    if not s["case"]["train"]:
        return dict(loss=nsp.distill_loss(s["logits"], s["top"], s["top_ids"], **kw))
    loss, dlogits = nsp.distill_grad(s["logits"], s["top"], s["top_ids"], weight=s["weight"], **kw)
    return dict(loss=loss, dlogits=dlogits)


def _own_route(s):
    nsp = _nsp()
    c = s["case"]
    r = nsp.route(s["logits"], c["k"], doc=s["doc"], normalize=c["normalize"])
    out = dict(ids=r.ids, weights=r.weights, counts=r.counts, tokens=r.tokens, loss=r.loss)
    if c["train"]:
        out["dlogits"] = nsp.route_backward(s["logits"], r, s["d_weights"], s["d_loss"],
                                            doc=s["doc"], normalize=c["normalize"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(scan=_own_scan, distill=_own_distill, route=_own_route)[op](state)
    return dict(scan=_plain_scan, distill=_plain_distill, route=_plain_route)[op](state)


# ---- what one pass cannot do without -------------------------------------------------
def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "scan":
        B, T, D = case["B"], case["T"], case["D"]
        n = B * T * D
        moved = 3 * es * n + 4 * D + 4 * B * D + (8 * B * T if case["packed"] else 0)
        moved += 4 * B * D if case["state"] else 0
        if case["train"]:  # dy in, dz and df out
            moved += 3 * es * n + 4 * D + (8 * B * D if case["state"] else 0)
        return dict(bytes=moved, flops=n * (30 if case["train"] else 10))
    if case["op"] == "distill":
        N, V, K = case["N"], case["V"], case["K"]
        moved = case["learned"] * N * (V * es + K * (4 + BYTES[case["tdtype"]])) + 4 * N
        moved += N if case["learned"] < 1 else 0
        moved += 4 * N if case["tail"] else 0
        if case["train"]:
            moved += N * V * es + 4 * N
        return dict(bytes=moved, flops=case["learned"] * N * V * (8 if case["train"] else 4))
    N, E, k = case["N"], case["E"], case["k"]
    moved = N * E * es + 8 * N * k + 4 * E + 8 + (4 * N if case["pad"] else 0)
    if case["train"]:
        moved += N * E * es + 4 * N * k + 4
    return dict(bytes=moved, flops=N * E * (12 if case["train"] else 6))


# ---- the definitions, in 64 bits --------------------------------------------------------
def _exact_scan(case, s):
    B, T, D = case["B"], case["T"], case["D"]
    f64 = dict(dtype=torch.float64, device=DEV)
    bias = torch.zeros(D, **f64) if s["bias"] is None else s["bias"].double()
    fresh = torch.zeros((B, T), dtype=torch.bool, device=DEV) if s["pos"] is None else s["pos"] == 0
    real = torch.ones_like(fresh) if s["doc"] is None else s["doc"] >= 0
    h = torch.zeros((B, D), **f64) if s["h0"] is None else s["h0"].double()
    y, before, gate = (torch.zeros((B, T, D), **f64) for _ in range(3))
    for t in range(T):
        prev = h.masked_fill(fresh[:, t, None], 0.0)
        a = 1.0 / (1.0 + torch.exp(-(s["f"][:, t].double() + bias)))
        new = a * prev + (1.0 - a) * s["z"][:, t].double()
        y[:, t] = new.masked_fill(~real[:, t, None], 0.0)
        h = torch.where(real[:, t, None], new, h)
        before[:, t], gate[:, t] = prev, a
    out = dict(y=y, h_last=h)
    if not case["train"]:
        return out
    up = torch.zeros((B, D), **f64) if s["dh"] is None else s["dh"].double()
    dz, df = torch.zeros((B, T, D), **f64), torch.zeros((B, T, D), **f64)
    for t in range(T - 1, -1, -1):
        d = up + s["dy"][:, t].double()
        a, ok = gate[:, t], real[:, t, None]
        dz[:, t] = ((1.0 - a) * d).masked_fill(~ok, 0.0)
        df[:, t] = (a * (1.0 - a) * d * (before[:, t] - s["z"][:, t].double())).masked_fill(~ok, 0.0)
        up = torch.where(ok, (a * d).masked_fill(fresh[:, t, None], 0.0), up)
    out.update(dz=dz, df=df, dbias=df.sum((0, 1)))
    if s["h0"] is not None:
        out["dh0"] = up
    return out


def _exact_distill(case, s):
    N, V, temp = case["N"], case["V"], case["temperature"]
    loss = torch.zeros(N, dtype=torch.float64, device=DEV)
    out = dict(loss=loss)
    if case["train"]:
        out["dlogits"] = torch.zeros((N, V), dtype=torch.float64, device=DEV)
    rows = max(1, (1 << 27) // V)
    for a in range(0, N, rows):
        x = s["logits"][a:a + rows].double() / temp
        log_q = torch.log_softmax(x, 1)
        t = s["top"][a:a + rows].double() / temp
        if s["lse"] is None:
            p = torch.softmax(t, 1)
        else:
            p = torch.exp(t - s["lse"][a:a + rows].double()[:, None])
        full = torch.zeros_like(x).scatter_add_(1, s["top_ids"][a:a + rows].long(), p)
        divergence = torch.special.xlogy(full, full) - full * log_q
        keep = torch.ones(len(x), dtype=torch.bool, device=DEV)
        if s["mask"] is not None:
            keep = s["mask"][a:a + rows] != 0
        loss[a:a + rows] = (temp * temp * divergence.sum(1)).masked_fill(~keep, 0.0)
        if case["train"]:
            g = temp * (full.sum(1, keepdim=True) * log_q.exp() - full)
            g *= s["weight"][a:a + rows].double()[:, None]
            out["dlogits"][a:a + rows] = g.masked_fill(~keep[:, None], 0.0)
    return out


def _exact_route(case, s):
    N, E, k = case["N"], case["E"], case["k"]
    x = s["logits"].double()
    real = torch.ones(N, dtype=torch.bool, device=DEV) if s["doc"] is None else s["doc"] >= 0
    p = torch.softmax(x, 1)
    left, columns, ids = x.clone(), torch.arange(E, device=DEV), []
    for _ in range(k):  # the largest that is left, the lowest index of equals
        best = torch.where(left == left.amax(1, keepdim=True), columns, E).amin(1)
        ids.append(best)
        left.scatter_(1, best[:, None], NEG_INF)
    ids = torch.stack(ids, 1)
    chosen = p.gather(1, ids)
    w = chosen / chosen.sum(1, keepdim=True) if case["normalize"] else chosen
    counts = torch.bincount(ids[real].reshape(-1), minlength=E).double()
    M = int(real.sum())
    coef = E / (k * max(1, M) ** 2)
    loss = coef * (counts * p[real].sum(0)).sum()
    out = dict(ids=ids.masked_fill(~real[:, None], -1).int(), weights=w * real[:, None],
               counts=counts.int(), tokens=torch.tensor(M, dtype=torch.int32), loss=loss)
    if not case["train"]:
        return out
    dw = s["d_weights"].double()
    d = p * counts * coef * s["d_loss"].double()
    d = d - p * d.sum(1, keepdim=True)
    soft = w if case["normalize"] else p  # the softmax that the weights come from
    at = w * dw
    part = torch.zeros_like(p).scatter_add_(1, ids, at)
    if case["normalize"]:
        soft = torch.zeros_like(p).scatter_add_(1, ids, w)
    d = d + part - soft * at.sum(1, keepdim=True)
    out["dlogits"] = d * real[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(scan=_exact_scan, distill=_exact_distill, route=_exact_route)[case["op"]](case, s)

"""The residual-stream operators: what is measured of them, and their plain forms.

Four operators at the ends of a transformer block, in the order in which a model meets them:

* ``lookup``   tokens -> rows of a table times a scale, h = scale * table[token], and with a norm its first RMSNorm
               y = h * rstd * gamma in the same call (the start of the residual stream);
* ``join``     block output x and stream r -> h = residual_scale * r + gate * (x * rstd_post * gamma_post) and
               y = h * rstd_pre * gamma_pre: the norm after a block, its gate, the scaled residual add and the norm
               before the next block;
* ``join_grad``    its gradients: dx, dr, dgamma_post, dgate, dgamma_pre;
* ``lookup_grad``  the table's gradient: row v is scale times the sum of the gradient rows of the tokens equal to v.

Cases are dicts: ``op``, ``n`` rows (tokens), ``h`` columns, ``dtype`` of the rows, ``wdtype`` of the parameters, and
per operator ``gates`` (0: no gate, 1: one gate vector for all rows, B > 1: one for each of B equal runs of rows),
``post`` (whether the block's output is normalised), ``vocab``, ``norm``, ``padding`` (an ignored token id, or -1).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
RESIDUAL_SCALE = 0.875  # what a depth-scaled residual stream keeps of itself at a block
EMBED_SCALE = 1.5
MOST_ROWS = 16384 * 4096  # n * h of the largest listed join
MOST_TABLE = 131072 * 4096  # vocab * h of the largest listed table


def listed():
    def join(name, op, n, h, dtype, wdtype, gates, post=True):
        return {"name": name, "op": op, "n": n, "h": h, "dtype": dtype, "wdtype": wdtype, "gates": gates, "post": post}

    def look(name, op, n, h, vocab, dtype, wdtype, norm=False, padding=-1):
        return {"name": name, "op": op, "n": n, "h": h, "vocab": vocab, "dtype": dtype, "wdtype": wdtype,
                "norm": norm, "padding": padding}

    return [
        # one new token of a served model: latency
        join("join 1x4096 bf16", "join", 1, 4096, "bf16", "bf16", 0),
        # a training step's activations with a learned gate for each channel (layer scale)
        join("join 8192x1024 bf16", "join", 8192, 1024, "bf16", "bf16", 1),
        # eight sequences of 2048 tokens, each with a gate of its own (conditioned blocks): the largest forward
        join("join 16384x4096 bf16", "join", 16384, 4096, "bf16", "bf16", 8),
        # ragged batch and width (rows neither 32- nor 16-byte aligned), no norm after the block
        join("join 1531x1001 f16", "join", 1531, 1001, "f16", "f32", 1, post=False),
        # the smallest training step
        join("join_grad 64x256 f32", "join_grad", 64, 256, "f32", "f32", 1),
        # a training step's gradients, the workload's non-power-of-two width
        join("join_grad 8192x5120 bf16", "join_grad", 8192, 5120, "bf16", "bf16", 1),
        # the widest rows
        join("join_grad 2048x16384 bf16", "join_grad", 2048, 16384, "bf16", "bf16", 0),
        # sequences of an odd length with gates of their own, fp32 parameters
        join("join_grad 7x1171x2056 f16", "join_grad", 7 * 1171, 2056, "f16", "f32", 7),
        # a decode step of eight sequences: the stream's first rows and their norm
        look("lookup 8x4096 bf16", "lookup", 8, 4096, 32768, "bf16", "bf16", norm=True),
        # a prompt or training batch, stream and first norm
        look("lookup 16384x4096 bf16", "lookup", 16384, 4096, 131072, "bf16", "bf16", norm=True),
        # the table's gradient of a small, padded, ragged batch with fp32 gradients
        look("lookup_grad 1999x1000 f16", "lookup_grad", 1999, 1000, 50001, "f16", "f32", padding=50000),
        # the table's gradient of a training batch: a dense gradient of a large vocabulary
        look("lookup_grad 16384x4096 bf16", "lookup_grad", 16384, 4096, 131072, "bf16", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["join", "join", "join_grad", "join_grad", "lookup", "lookup_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    wdtype = rng.choice([dtype, "f32"])
    h = _log_int(rng, 64, 16384)
    step = rng.choice([1, 8, 16, 16, 128])  # odd widths, 16- and 32-byte rows, whole tiles
    h = max(step, h // step * step)
    # fp32 rows take twice the bytes, a gradient reads and writes more tensors: fewer rows
    cost = (2 if dtype == "f32" else 1) * (2 if op == "join_grad" else 1)
    n = _log_int(rng, 1, max(1, min(32768, MOST_ROWS // (h * cost))))
    case = {"op": op, "n": n, "h": h, "dtype": dtype, "wdtype": wdtype}
    if op in ("join", "join_grad"):
        gates = rng.choice([0, 1, 1, 2])
        if gates == 2:
            gates = min(n, rng.choice([2, 3, 8, 13]))
            n = n // gates * gates
        case.update(n=n, gates=gates, post=rng.random() < 0.75)
    else:
        vocab = _log_int(rng, 64, max(64, min(131072, MOST_TABLE // (h * (4 if "f32" in (dtype, wdtype) else 1)))))
        case.update(vocab=vocab, norm=op == "lookup" and rng.random() < 0.7,
                    padding=vocab - 1 if op == "lookup_grad" and rng.random() < 0.4 else -1)
    return case


def _normal(shape, gen, dtype, mean=0.0, std=1.0):
    t = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(mean, std, generator=gen)
    return t.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    n, h, dt, wt = case["n"], case["h"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
    s = dict(case)
    if case["op"] in ("join", "join_grad"):
        s["x"] = _normal((n, h), gen, dt, std=0.7)  # the block's output
        s["r"] = _normal((n, h), gen, dt, std=2.0)  # the residual stream
        s["gpost"] = _normal((h,), gen, wt, mean=1.0, std=0.1)
        s["gpre"] = _normal((h,), gen, wt, mean=1.0, std=0.1)
        g = case["gates"]
        s["gate"] = None if g == 0 else _normal((h,) if g == 1 else (g, h), gen, wt, mean=0.5, std=0.25)
        if case["op"] == "join_grad":
            s["dy"] = _normal((n, h), gen, dt)
            s["dh"] = _normal((n, h), gen, dt, std=0.5)  # what arrives through the stream
            # what the forward left behind: the stored stream (here r) and both reciprocal norms
            s["rpost"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float() if case["post"] else None
            s["rpre"] = (s["r"].double().square().mean(1) + EPS).rsqrt().float()
    else:
        # word frequencies fall as 1/rank
        u = torch.empty(n, device="cuda", dtype=torch.float64).uniform_(0.0, 1.0, generator=gen)
        tokens = torch.exp(u * math.log(case["vocab"] + 1)).long().sub_(1).clamp_(0, case["vocab"] - 1)
        if case["padding"] >= 0:  # a padded batch: about a fifth of the positions
            pad = torch.empty(n, device="cuda").uniform_(0.0, 1.0, generator=gen) < 0.2
            tokens[pad] = case["padding"]
        s["tokens"] = tokens
        if case["op"] == "lookup":
            s["table"] = _normal((case["vocab"], h), gen, dt)
            s["gamma"] = _normal((h,), gen, wt, mean=1.0, std=0.1)
        else:
            s["dh"] = _normal((n, h), gen, dt)
    return s


# ----------------------------------------------------------------------------- plain forms, 32 bits

def _gate_rows(gate, n):
    """The gate of each row: a vector broadcasts, B vectors serve n / B rows each."""
    gate = gate.float()
    return gate if gate.dim() == 1 else gate.repeat_interleave(n // gate.shape[0], 0)


def _join(s):
    dt = s["x"].dtype
    p, rpost = s["x"].float(), None
    if s["post"]:
        rpost = 1.0 / torch.sqrt((p * p).mean(1) + EPS)
        p = p * rpost[:, None] * s["gpost"].float()
    if s["gate"] is not None:
        p = p * _gate_rows(s["gate"], s["n"])
    hs = RESIDUAL_SCALE * s["r"].float() + p
    rpre = 1.0 / torch.sqrt((hs * hs).mean(1) + EPS)
    y = hs * rpre[:, None] * s["gpre"].float()
    return y.to(dt), hs.to(dt), rpost, rpre


def _join_grad(s):
    n, h = s["n"], s["h"]
    dt = s["x"].dtype
    wt = s["gpost"].dtype
    dy, hs, x = s["dy"].float(), s["r"].float(), s["x"].float()
    gate = 1.0 if s["gate"] is None else _gate_rows(s["gate"], n)
    xh = hs * s["rpre"][:, None]
    g = dy * s["gpre"].float()
    dh = s["dh"].float() + s["rpre"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    dgpre = (dy * xh).sum(0)
    dr = RESIDUAL_SCALE * dh
    if s["post"]:
        oh = x * s["rpost"][:, None]
        dgate = dh * (oh * s["gpost"].float())
        dp = dh * gate
        dgpost = (dp * oh).sum(0).to(wt)
        g = dp * s["gpost"].float()
        dx = s["rpost"][:, None] * (g - oh * (g * oh).mean(1, keepdim=True))
    else:
        dgate, dgpost = dh * x, None
        dx = dh * gate
    if s["gate"] is None:
        dgate = None
    elif s["gate"].dim() == 1:
        dgate = dgate.sum(0).to(wt)
    else:
        dgate = dgate.view(s["gates"], n // s["gates"], h).sum(1).to(wt)
    return dx.to(dt), dr.to(dt), dgpost, dgate, dgpre.to(wt)


def _lookup(s):
    hs = s["table"][s["tokens"]].float() * EMBED_SCALE
    dt = s["table"].dtype
    if not s["norm"]:
        return hs.to(dt)
    rstd = 1.0 / torch.sqrt((hs * hs).mean(1) + EPS)
    return (hs * rstd[:, None] * s["gamma"].float()).to(dt), hs.to(dt), rstd


def _lookup_grad(s):
    rows = s["dh"].float() * EMBED_SCALE
    if s["padding"] >= 0:
        rows = rows * (s["tokens"] != s["padding"])[:, None]
    grad = torch.zeros(s["vocab"], s["h"], device=rows.device, dtype=torch.float32)
    return grad.index_add_(0, s["tokens"], rows).to(DTYPES[s["wdtype"]])


# ----------------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        import rmsnorm_ln_fwd_gb300 as nl

        if op == "join":
            return nl.sandwich_rms(s["x"], s["r"], s["gpost"] if s["post"] else None, s["gate"], s["gpre"], EPS,
                                   residual_scale=RESIDUAL_SCALE, post_norm=s["post"])
        if op == "join_grad":
            return nl.sandwich_rms_grad(s["dy"], s["x"], s["r"], s["rpost"], s["rpre"],
                                        s["gpost"] if s["post"] else None, s["gate"], s["gpre"], s["dh"],
                                        residual_scale=RESIDUAL_SCALE)
        if op == "lookup":
            if s["norm"]:
                return nl.embedding_rms(s["tokens"], s["table"], s["gamma"], EPS, EMBED_SCALE)
            return nl.embedding_lookup(s["tokens"], s["table"], EMBED_SCALE)
        return nl.embedding_grad(s["dh"], s["tokens"], s["vocab"], EMBED_SCALE,
                                 padding_idx=s["padding"] if s["padding"] >= 0 else None,
                                 param_dtype=DTYPES[s["wdtype"]])
    return {"join": _join, "join_grad": _join_grad, "lookup": _lookup, "lookup_grad": _lookup_grad}[op](s)


def work(case):
    n, h, e, ew = case["n"], case["h"], BYTES[case["dtype"]], BYTES[case["wdtype"]]
    op = case["op"]
    if op == "join":  # x, r in; h, y out
        vectors = (2 if case["post"] else 1) + case["gates"]
        return {"bytes": 4 * n * h * e + vectors * h * ew + (8 if case["post"] else 4) * n, "flops": 9 * n * h}
    if op == "join_grad":  # dy, dh, h, x in; dx, dr out; each parameter in and its gradient out
        vectors = (2 if case["post"] else 1) + case["gates"]
        return {"bytes": 6 * n * h * e + 2 * vectors * h * ew + (8 if case["post"] else 4) * n, "flops": 24 * n * h}
    # each distinct row of the table is read once: with frequencies of 1/rank about this many are
    v = case["vocab"]
    if op == "lookup":
        ranks = math.log(v + 1)
        distinct = sum(1.0 - (1.0 - math.log1p(1.0 / k) / ranks) ** n for k in range(1, v + 1))
        out = 2 if case["norm"] else 1
        return {"bytes": 8 * n + (distinct + out * n) * h * e + ((h * ew + 4 * n) if case["norm"] else 0),
                "flops": (5 if case["norm"] else 1) * n * h}
    kept = 1.0 if case["padding"] < 0 else 0.8
    return {"bytes": 8 * n + kept * n * h * e + v * h * ew, "flops": 2 * n * h}


# ----------------------------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    n, h = s["n"], s["h"]

    def d(name):
        return s[name].to(torch.float64)

    def norm(v, gamma):
        rms = torch.linalg.vector_norm(v, dim=1, keepdim=True).square().div_(h).add_(EPS).sqrt_()
        return v / rms * gamma, (1.0 / rms).squeeze(1)

    def mean_with(a, b):
        return torch.einsum("nh,nh->n", a, b).div_(h)[:, None]

    if s["op"] == "join":
        p, rpost = norm(d("x"), d("gpost")) if s["post"] else (d("x"), None)
        if s["gate"] is not None:
            runs = s["gate"].double().view(-1, 1, h)
            p = (p.view(runs.shape[0], -1, h) * runs).reshape(n, h)
        hs = d("r").mul_(RESIDUAL_SCALE).add_(p)
        y, rpre = norm(hs, d("gpre"))
        return y, hs, rpost, rpre
    if s["op"] == "join_grad":
        runs = 1 if s["gate"] is None else s["gate"].double().view(-1, 1, h)
        b = 1 if s["gate"] is None else runs.shape[0]

        def gated(v):
            return (v.view(b, -1, h) * runs).reshape(n, h)

        rpre = d("rpre")[:, None]
        dxh = d("dy") * d("gpre")
        xh = d("r") * rpre
        dh = d("dh") + rpre * dxh - rpre * xh * mean_with(dxh, xh)
        dgpre = torch.einsum("nh,nh->h", d("dy"), xh)
        rpost = d("rpost")[:, None] if s["post"] else 1.0
        oh = d("x") * rpost
        by_run = torch.einsum("bth,bth->bh", dh.view(b, -1, h), oh.view(b, -1, h))  # sums of dh * x_hat of each run
        dgate = None
        if s["gate"] is not None:
            dgate = (by_run * (d("gpost") if s["post"] else 1.0)).view(s["gate"].shape)
        dgpost = None
        dx = gated(dh)
        if s["post"]:
            dgpost = (by_run * (1.0 if s["gate"] is None else runs.view(b, h))).sum(0)
            dx = dx * d("gpost")
            dx = rpost * (dx - oh * mean_with(dx, oh))
        return dx, dh * RESIDUAL_SCALE, dgpost, dgate, dgpre
    if s["op"] == "lookup":
        hs = torch.nn.functional.one_hot(s["tokens"], s["vocab"]).double() @ d("table") * EMBED_SCALE \
            if n * s["vocab"] <= 1 << 20 else torch.gather(d("table"), 0, s["tokens"][:, None].expand(n, h)) * EMBED_SCALE
        if not s["norm"]:
            return hs
        y, rstd = norm(hs, d("gamma"))
        return y, hs, rstd
    keep = s["tokens"] != s["padding"]
    order = torch.argsort(s["tokens"][keep], stable=True)
    ids, counts = torch.unique_consecutive(s["tokens"][keep][order], return_counts=True)
    grad = torch.zeros(s["vocab"], h, device="cuda", dtype=torch.float64)
    if ids.numel():
        ends = counts.cumsum(0)
        owner = torch.repeat_interleave(torch.arange(ids.numel(), device="cuda"), counts)
        sums = torch.zeros(ids.numel(), h, device="cuda", dtype=torch.float64)
        assert int(ends[-1]) == owner.numel()
        sums.scatter_add_(0, owner[:, None].expand(-1, h), d("dh")[keep][order])
        grad[ids] = sums * EMBED_SCALE
    return grad

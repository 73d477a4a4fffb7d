"""The operators inside the attention block and at the end of a residual stream: what is measured of them, and their
plain forms.

Four operators, two pairs of a forward and its gradient:

* ``rotary``         the RMSNorm of each head of the queries and keys, and the rotation by their tokens' positions:
                     n = x * rstd * gamma for each head, then in each pair (a, b) of its first ``rot`` columns
                     y_a = n_a * cos - n_b * sin, y_b = n_b * cos + n_a * sin;
* ``rotary_grad``    its gradients: dq, dk, dgamma_q, dgamma_k;
* ``logprob``        rows of logits and a token for each -> log probability of the token, entropy of the row, its
                     log of summed exponentials and statistics, and the ``top`` most probable tokens;
* ``logprob_grad``   the gradient of the logits from those of log probability, entropy and log-sum-exp.

Cases are dicts: ``op`` and ``dtype``; for the rotation ``b`` sequences of ``t`` tokens, ``hq`` and ``hk`` heads of
``d`` columns, ``rot`` rotated ones, ``pairs`` (halves or interleaved), ``wdtype`` of gamma, ``table`` rows of cos and
sin, ``packed`` (positions given for each token) and ``fused`` (q and k are parts of one projection's output); for the
logits ``n`` rows of ``v``, ``banned`` columns at -inf behind the vocabulary, ``top``, ``scale``, ``ignore`` (a share of
the rows has no token) and for the gradient ``with_entropy`` and ``with_lse``.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
BASE = 10000.0  # of the rotation's angles
IGNORE = -100
MOST_HEADS = 16384 * 40 * 128  # elements of q and k together of the largest listed rotation
MOST_LOGITS = 4096 * 131072  # elements of the largest listed logits (half precision)


def listed():
    def rotary(name, op, b, t, hq, hk, d, rot, dtype, wdtype, pairs="halves", packed=False, fused=True, table=8192):
        return {"name": name, "op": op, "b": b, "t": t, "hq": hq, "hk": hk, "d": d, "rot": rot, "dtype": dtype,
                "wdtype": wdtype, "pairs": pairs, "packed": packed, "fused": fused, "table": table}

    def logits(name, op, n, v, dtype, scale=1.0, top=0, banned=0, ignore=False, with_entropy=True, with_lse=False):
        return {"name": name, "op": op, "n": n, "v": v, "dtype": dtype, "scale": scale, "top": top, "banned": banned,
                "ignore": ignore, "with_entropy": with_entropy, "with_lse": with_lse}

    return [
        # decode: one new token of each of eight sequences, at positions of their own: latency
        rotary("rotary 8x1 32+8x128 bf16", "rotary", 8, 1, 32, 8, 128, 128, "bf16", "bf16", packed=True),
        # a training batch or a long prompt
        rotary("rotary 4x4096 32+8x128 bf16", "rotary", 4, 4096, 32, 8, 128, 128, "bf16", "bf16"),
        # a ragged batch packed into one row of tokens, part of a head rotated, pairs beside each other
        rotary("rotary 1x1531 12+4x80 f16", "rotary", 1, 1531, 12, 4, 80, 32, "f16", "f32", "interleaved", packed=True),
        # the gradients of a training batch
        rotary("rotary_grad 4x2048 32+8x128 bf16", "rotary_grad", 4, 2048, 32, 8, 128, 128, "bf16", "bf16"),
        # gradients of sequences of an odd length, as many key heads as query heads, in fp32
        rotary("rotary_grad 7x333 16+16x64 f32", "rotary_grad", 7, 333, 16, 16, 64, 64, "f32", "f32", fused=False),
        # the gradients of a small ragged batch
        rotary("rotary_grad 1x517 9+3x96 f16", "rotary_grad", 1, 517, 9, 3, 96, 48, "f16", "f32", packed=True),
        # decode: one token's distribution with its alternatives, a large vocabulary
        logits("logprob 1x131072 bf16 top 20", "logprob", 1, 131072, "bf16", top=20),
        # a batch of answers with a temperature and alternatives, an odd vocabulary
        logits("logprob 333x50001 f16 top 5", "logprob", 333, 50001, "f16", scale=1.25, top=5),
        # a training batch over a padded vocabulary
        logits("logprob 4096x131072 bf16", "logprob", 4096, 131072, "bf16", banned=96, ignore=True),
        # its gradient, with an entropy term: the largest
        logits("logprob_grad 4096x131072 bf16", "logprob_grad", 4096, 131072, "bf16", banned=96, ignore=True),
        # fp32 logits with a term in the log-sum-exp
        logits("logprob_grad 777x32000 f32", "logprob_grad", 777, 32000, "f32", with_entropy=False, with_lse=True),
        # a small batch of an odd vocabulary
        logits("logprob_grad 16x50001 f16", "logprob_grad", 16, 50001, "f16", scale=0.8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "logprob", "logprob_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    wide = 2 if dtype == "f32" else 1
    if op in ("rotary", "rotary_grad"):
        d = rng.choice([64, 80, 96, 112, 128, 128, 128, 192, 256])
        hk = rng.choice([1, 2, 3, 4, 8, 8, 16])
        hq = hk * rng.choice([1, 2, 4, 5, 8])
        cost = wide * (2 if op == "rotary_grad" else 1)
        n = _log_int(rng, 1, min(65536, MOST_HEADS // ((hq + hk) * d * cost)))
        b = rng.choice([1, 1, 2, 4, 7])
        t = max(1, min(8192, n // b))
        return {"op": op, "b": b, "t": t, "hq": hq, "hk": hk, "d": d, "rot": rng.choice([d, d, d // 2]), "dtype": dtype,
                "wdtype": rng.choice([dtype, "f32"]), "pairs": rng.choice(["halves", "halves", "interleaved"]),
                "packed": rng.random() < 0.5, "fused": rng.random() < 0.6, "table": 8192}
    v = _log_int(rng, 512, 262144)
    step = rng.choice([1, 16, 128, 128])  # odd vocabularies, padded ones
    v = max(step, v // step * step)
    n = _log_int(rng, 1, min(16384, MOST_LOGITS // (v * wide)))
    top = rng.choice([0, 0, 1, 5, 20]) if op == "logprob" else 0
    if top:
        n = min(n, 1024)  # a server's batch
    return {"op": op, "n": n, "v": v, "dtype": dtype, "scale": rng.choice([1.0, 1.0, 0.8, 1.25]), "top": top,
            "banned": rng.choice([0, 0, min(64, v // 8)]), "ignore": rng.random() < 0.4,
            "with_entropy": rng.random() < 0.6, "with_lse": rng.random() < 0.4}


def _normal(shape, gen, dtype, mean=0.0, std=1.0):
    t = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(mean, std, generator=gen)
    return t.to(dtype)


def _heads(b, t, hq, hk, d, fused, gen, dtype, std):
    """q (b, t, hq, d) and k (b, t, hk, d): parts of one projection's output with the values behind them, or tensors of
    their own."""
    if not fused:
        return _normal((b, t, hq, d), gen, dtype, std=std), _normal((b, t, hk, d), gen, dtype, std=std)
    whole = _normal((b, t, (hq + 2 * hk) * d), gen, dtype, std=std)
    q, k, _ = whole.split([hq * d, hk * d, hk * d], -1)
    return q.unflatten(-1, (hq, d)), k.unflatten(-1, (hk, d))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("rotary", "rotary_grad"):
        b, t, hq, hk, d, rot = (case[k] for k in ("b", "t", "hq", "hk", "d", "rot"))
        wt = DTYPES[case["wdtype"]]
        s["q"], s["k"] = _heads(b, t, hq, hk, d, case["fused"], gen, dt, 1.5)
        s["gq"] = _normal((d,), gen, wt, mean=1.0, std=0.1)
        s["gk"] = _normal((d,), gen, wt, mean=1.0, std=0.1)
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * \
            BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = None
        if case["packed"]:  # sequences that start anywhere in the table: each at a place of its own, then in order
            at = torch.randint(0, case["table"], (b, 1), device="cuda", generator=gen)
            s["positions"] = (at + torch.arange(t, device="cuda")) % case["table"]
        if case["op"] == "rotary_grad":
            s["dyq"], s["dyk"] = _heads(b, t, hq, hk, d, False, gen, dt, 1.0)
        return s
    n, v = case["n"], case["v"]
    z = _normal((n, v), gen, dt, std=2.5)
    tokens = torch.randint(0, v - case["banned"], (n,), device="cuda", generator=gen)
    z[torch.arange(n, device="cuda"), tokens] += _normal((n,), gen, dt, mean=6.0, std=4.0)  # mostly probable tokens
    if case["banned"]:
        z[:, v - case["banned"]:] = -math.inf
    if case["ignore"]:
        tokens[torch.empty(n, device="cuda").uniform_(0.0, 1.0, generator=gen) < 0.1] = IGNORE
    s["z"], s["tokens"] = z, tokens
    if case["op"] == "logprob_grad":
        m, l, h = _statistics64(z, case["scale"])
        s["stats"] = torch.stack([m, l], 1).float()
        s["entropy"] = h.float() if case["with_entropy"] else None
        s["dlogprob"] = _normal((n,), gen, torch.float32)
        s["dentropy"] = _normal((n,), gen, torch.float32, std=0.1) if case["with_entropy"] else None
        s["dlse"] = _normal((n,), gen, torch.float32, std=0.1) if case["with_lse"] else None
    return s


def _statistics64(z, scale):
    """Maximum, log of the sum of exp(scale * (z - maximum)) and entropy of each row, in 64 bits, some rows at a time."""
    out = []
    for part in z.split(max(1, (1 << 26) // z.shape[1])):
        part = part.double()
        m = part.amax(1)
        x = part.sub_(m[:, None]).mul_(scale)
        p = x.exp()
        total = p.sum(1)
        out.append(torch.stack([m, total.log(), total.log() - p.mul_(x.clamp_(min=-1e4)).sum(1) / total]))
    return torch.cat(out, 1)


# ----------------------------------------------------------------------------- plain forms, 32 bits

def _tables(s):
    """cos and sin of each token, (b or 1, t, 1, rot / 2)."""
    p = s["positions"] if s["positions"] is not None else torch.arange(s["t"], device=s["q"].device)[None]
    return s["cos"][p][:, :, None], s["sin"][p][:, :, None]


def _turn(x, cos, sin, s):
    """Every pair of x's first rot columns turned by its token's angle."""
    rot = s["rot"]
    if s["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _rotary(s):
    cos, sin = _tables(s)

    def one(x, gamma):
        f = x.float()
        rstd = 1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
        return _turn(f * rstd * gamma.float(), cos, sin, s).to(x.dtype)

    return one(s["q"], s["gq"]), one(s["k"], s["gk"])


def _rotary_grad(s):
    cos, sin = _tables(s)

    def one(dy, x, gamma):
        f = x.float()
        rstd = 1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
        u = _turn(dy.float(), cos, -sin, s)
        xh = f * rstd
        w = u * gamma.float()
        dx = rstd * (w - xh * (w * xh).mean(-1, keepdim=True))
        return dx.to(x.dtype), (u * xh).sum((0, 1, 2)).to(gamma.dtype)

    dq, dgq = one(s["dyq"], s["q"], s["gq"])
    dk, dgk = one(s["dyk"], s["k"], s["gk"])
    return dq, dk, dgq, dgk


def _logprob(s):
    z = s["z"].float()
    n, v = z.shape
    m = z.amax(1)
    x = (z - m[:, None]) * s["scale"]
    p = torch.exp(x)
    total = p.sum(1)
    log_sum = torch.log(total)
    entropy = None
    if s["with_entropy"]:
        entropy = log_sum - torch.where(p > 0, p * x, 0.0).sum(1) / total
    valid = s["tokens"] != IGNORE
    at = torch.where(valid, s["tokens"], 0)
    logprob = torch.where(valid, x.gather(1, at[:, None])[:, 0] - log_sum, 0.0)
    lse = s["scale"] * m + log_sum
    stats = torch.stack([m, log_sum], 1)
    if not s["top"]:
        return logprob, entropy, lse, stats
    # descending logits, equal ones by id: the value's bits in an order of whole numbers, then the id
    bits = z.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 32) + ((1 << 32) - 1 - torch.arange(v, device=z.device))
    ids = (1 << 32) - 1 - (key.topk(s["top"], 1).values & 0xffffffff)
    return logprob, entropy, lse, stats, x.gather(1, ids) - log_sum[:, None], ids


def _logprob_grad(s):
    z = s["z"].float()
    m, log_sum = s["stats"][:, :1], s["stats"][:, 1:]
    logp = (z - m) * s["scale"] - log_sum
    p = torch.exp(logp)
    valid = s["tokens"] != IGNORE
    dlogprob = torch.where(valid, s["dlogprob"], 0.0)
    coefficient = -dlogprob[:, None]
    if s["dlse"] is not None:
        coefficient = coefficient + s["dlse"][:, None]
    if s["dentropy"] is not None:
        coefficient = coefficient - s["dentropy"][:, None] * (logp + s["entropy"][:, None])
    grad = torch.where(p > 0, p * coefficient, 0.0)
    grad.scatter_add_(1, torch.where(valid, s["tokens"], 0)[:, None], dlogprob[:, None])
    return (grad * s["scale"]).to(s["z"].dtype)


# ----------------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        import rmsnorm_ln_fwd_gb300 as nl

        if op == "rotary":
            return nl.head_rms_rotary(s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"], s["positions"], EPS,
                                      interleaved=s["pairs"] == "interleaved")
        if op == "rotary_grad":
            return nl.head_rms_rotary_grad(s["dyq"], s["dyk"], s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"],
                                           s["positions"], EPS, interleaved=s["pairs"] == "interleaved")
        if op == "logprob":
            out = nl.token_logprobs(s["z"], s["tokens"], s["scale"], top=s["top"], ignore_index=IGNORE,
                                    entropy=s["with_entropy"])
            return out if s["top"] else out[:4]
        return nl.token_logprobs_grad(s["dlogprob"], s["z"], s["tokens"], s["stats"], s["entropy"], s["dentropy"],
                                      s["dlse"], s["scale"], ignore_index=IGNORE)
    return {"rotary": _rotary, "rotary_grad": _rotary_grad, "logprob": _logprob, "logprob_grad": _logprob_grad}[op](s)


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("rotary", "rotary_grad"):
        n, heads, d = case["b"] * case["t"], case["hq"] + case["hk"], case["d"]
        tables = min(case["table"], n if case["packed"] else case["t"]) * case["rot"] * 4 + (8 * n if case["packed"] else 0)
        gammas = 2 * d * BYTES[case["wdtype"]]
        if case["op"] == "rotary":  # q, k in and out
            return {"bytes": 2 * n * heads * d * e + tables + gammas, "flops": 10 * n * heads * d}
        # q, k and their outputs' gradients in, their gradients out
        return {"bytes": 3 * n * heads * d * e + tables + 2 * gammas, "flops": 20 * n * heads * d}
    n, v = case["n"], case["v"]
    if case["op"] == "logprob":
        out = 4 * (4 + (1 if case["with_entropy"] else 0)) + 12 * case["top"]
        return {"bytes": n * v * e + n * (8 + out), "flops": 6 * n * v}
    rows = 8 + 8 + 4 + (8 if case["with_entropy"] else 0) + (4 if case["with_lse"] else 0)
    return {"bytes": 2 * n * v * e + n * rows, "flops": 7 * n * v}


# ----------------------------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("rotary", "rotary_grad"):
        rot, half = s["rot"], s["rot"] // 2
        p = s["positions"] if s["positions"] is not None else torch.arange(s["t"], device="cuda").expand(s["b"], -1)
        unit = torch.complex(s["cos"].double(), s["sin"].double())[p.flatten()].view(s["b"], s["t"], 1, half)

        def forward(x, gamma):
            n = torch.nn.functional.rms_norm(x, (s["d"],), gamma, EPS)
            head = n[..., :rot]
            pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if s["pairs"] == "halves" else head.unflatten(-1, (half, 2))
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
            turned = turned.transpose(-1, -2).flatten(-2) if s["pairs"] == "halves" else turned.flatten(-2)
            return torch.cat([turned, n[..., rot:]], -1)

        if s["op"] == "rotary":
            return forward(s["q"].double(), s["gq"].double()), forward(s["k"].double(), s["gk"].double())
        leaves = [s[name].double().requires_grad_() for name in ("q", "k", "gq", "gk")]
        return torch.autograd.grad([forward(leaves[0], leaves[2]), forward(leaves[1], leaves[3])], leaves,
                                   [s["dyq"].double(), s["dyk"].double()])
    a, rows = s["scale"], max(1, (1 << 26) // s["v"])
    if s["op"] == "logprob":
        parts = []
        for z, tokens in zip(s["z"].split(rows), s["tokens"].split(rows)):
            logp = torch.log_softmax(z.double() * a, 1)
            lse = torch.logsumexp(z.double() * a, 1)
            m = z.amax(1).double()
            has = tokens != IGNORE
            part = [torch.zeros_like(lse), torch.special.entr(logp.exp()).sum(1), lse, torch.stack([m, lse - a * m], 1)]
            part[0][has] = logp[has, tokens[has]]
            if s["top"]:
                order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :s["top"]]
                part += [logp.gather(1, order), order]
            parts.append(part)
        out = [torch.cat(x) for x in zip(*parts)]
        return out if s["with_entropy"] else [out[0], None, *out[2:]]
    parts = []
    for i in range(0, s["n"], rows):
        z, tokens = s["z"][i:i + rows].double().requires_grad_(), s["tokens"][i:i + rows]
        logp = torch.log_softmax(z * a, 1)
        at = tokens.clamp(min=0)[:, None]
        loss = (logp.gather(1, at)[:, 0] * s["dlogprob"][i:i + rows] * (tokens != IGNORE)).sum()
        if s["with_entropy"]:
            entropy = -(logp.exp() * logp.masked_fill(logp == -math.inf, 0.0)).sum(1)
            loss = loss + (entropy * s["dentropy"][i:i + rows]).sum()
        if s["with_lse"]:
            loss = loss + (torch.logsumexp(z * a, 1) * s["dlse"][i:i + rows]).sum()
        parts.append(torch.autograd.grad(loss, z)[0])
    return torch.cat(parts)

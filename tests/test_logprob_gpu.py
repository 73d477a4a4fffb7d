"""Log probabilities of given tokens and the logits' gradient on the GPU against
the fp64 oracle, and both ends of the stream together.

Tolerances, from the arithmetic (U = 2^-24, half an fp32 step; x = scale (z - m)):

* an exponential: its argument in powers of two is a difference, the scale's
  product with log2(e) and a product, 4 steps of U of |x| in all; ex2 adds 4 U.
  Reference changes (a thread's own, the thread's to the CTA's, the CTA's to the
  row's) multiply it by such exponentials again, whose arguments add up to less
  than |x| + 24: (8 |x| + 64) U.
* their sum: at most V / 512 additions in a thread (256 a row, with two sums each;
  or 128 in one of fewer threads with 16 chunks of 16 or fewer) and 136 in all
  besides.  So log(sum) is off by U (8 E|x| + 200 + V / 512) with E the mean under p,
  and by two steps of its own.
* logprob = x_t - log(sum): 4 U |x_t| more.  lse: the product's and sum's steps.
* entropy = log(sum) - E[x]: the sum of e x has each term's error and |x| U more.
* the gradient's p: (8 |x| + 4 |log sum| + 24) U with the coefficients' steps.
"""

import numpy as np
import pytest
import torch

import rmsnorm_ln_fwd_gb300 as nl
from oracle import head_oracle as O
from rmsnorm_ln_fwd_gb300 import _lib, synth
from test_heads_gpu import close, n64, rnd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_ln_fwd_gb300 import _build
    _build.build()
    _lib.device_errors()


def make(N, V, dt, seed=0, std=2.5, banned=0.0, ignore=None):
    z = rnd((N, V), seed, DT[dt], std=std)
    r = np.random.default_rng(seed)
    tokens = torch.tensor(r.integers(0, V, N), device=DEV)
    if banned:
        z[torch.tensor(r.random((N, V)) < banned, device=DEV)] = -INF
    if ignore is not None:
        tokens[torch.tensor(r.random(N) < 0.2, device=DEV)] = ignore
    return z, tokens


def same_or_close(got, ref, slack, what):
    """As close; infinities have to be the same ones."""
    g = n64(got).reshape(np.shape(ref))
    inf = np.isinf(ref)
    assert np.array_equal(g[inf], ref[inf]), what
    ok = ~inf
    close(got.reshape(np.shape(ref))[torch.tensor(ok, device=got.device)], ref[ok], np.broadcast_to(slack, ref.shape)[ok], what)


def check(z, tokens, scale, out, top=0, ignore=None, entropy=True):
    logprob, ent, lse, stats, tlp, tid = out
    V = z.shape[-1]
    Z, tk = n64(z).reshape(-1, V), None if tokens is None else tokens.cpu().numpy().reshape(-1)
    rlp, rent, rlse, rm, rl, x, p = O.logprob_forward(Z, tk, scale, ignore)
    ax = np.where(np.isinf(x), 0.0, np.abs(x))
    E1, E2 = (p * ax).sum(1), (p * ax * ax).sum(1)
    fin = np.isfinite(rl)
    # (1 + 4 U) covers what is of second order in U
    dl = U * (8 * E1 + 200 + V / 512 + 2 * np.abs(np.where(fin, rl, 0.0))) * (1 + 4 * U)
    st = n64(stats).reshape(-1, 2)
    assert np.array_equal(st[:, 0], rm)
    same_or_close(stats.reshape(-1, 2)[:, 1], rl, dl, "log_sum")
    same_or_close(lse, rlse, dl + 2 * U * np.abs(np.where(fin, scale * rm, 0.0)), "lse")
    if tokens is None:
        assert logprob is None
    else:
        has = O.has_token(tk, V, ignore)
        xt = np.where(has, np.take_along_axis(ax, np.where(has, tk, 0)[:, None], 1)[:, 0], 0.0)
        same_or_close(logprob, rlp, np.where(has, dl + 4 * U * xt, 0.0), "logprob")
    if entropy:
        same_or_close(ent, rent, dl * (1 + E1) + U * (9 * E2 + (206 + V / 512) * E1), "entropy")
    else:
        assert ent is None
    if top:
        want = O.top_ids(Z, top)
        got = tid.cpu().numpy().reshape(-1, top)
        assert tid.dtype == torch.int64 and np.array_equal(got, want)
        with np.errstate(invalid="ignore"):
            xx = np.where(want < 0, -np.inf, np.take_along_axis(x, np.maximum(want, 0), 1) - rl[:, None])
        xa = np.take_along_axis(ax, np.maximum(want, 0), 1)
        same_or_close(tlp.reshape(-1, top), xx, dl[:, None] + 4 * U * xa, "top_logprobs")
    else:
        assert tlp is None and tid is None


def check_grad(z, tokens, scale, got, stats, ent, dlp, dent, dlse, ignore=None):
    V = z.shape[-1]
    Z, st = n64(z).reshape(-1, V), n64(stats).reshape(-1, 2)
    tk = None if tokens is None else tokens.cpu().numpy().reshape(-1)
    v = [None if t is None else n64(t).reshape(-1) for t in (dlp, ent, dent, dlse)]
    ref = O.logprob_backward(v[0], Z, tk, st[:, 0], st[:, 1], v[1], v[2], v[3], scale, ignore)
    m, l = st[:, :1], st[:, 1:]
    with np.errstate(invalid="ignore"):
        x = np.abs(scale * (Z - m))
        logp = scale * (Z - m) - l
    x, p = np.where(np.isfinite(x), x, 0.0), np.where(np.isneginf(l), 0.0, np.exp(np.where(np.isnan(logp), -np.inf, logp)))
    C = np.zeros((Z.shape[0], 1))
    own = np.zeros_like(Z)
    if v[0] is not None:
        has = O.has_token(tk, V, ignore)
        C = C + np.abs(np.where(has, v[0], 0.0))[:, None]
        own[np.arange(len(tk))[has], tk[has]] = np.abs(v[0][has])
    if v[3] is not None:
        C = C + np.abs(v[3])[:, None]
    if v[2] is not None:
        C = C + np.abs(v[2])[:, None] * (np.abs(v[1])[:, None] + np.where(np.isfinite(logp), np.abs(logp), 0.0))
    al = np.where(np.isfinite(l), np.abs(l), 0.0)
    slack = scale * (p * C * (8 * x + 4 * al + 24) * U + 4 * U * own + 2.0 ** -126 * C)
    close(got, ref.reshape(got.shape), slack.reshape(got.shape), "dlogits")


def grads_in(N, seed):
    return [rnd((N,), seed + i, torch.float32, std=s) for i, s in enumerate((1.0, 0.3, 0.3))]


SHAPES = [(1, 1), (1, 2), (3, 7), (2, 33), (5, 513), (40, 1000), (1, 4097), (7, 8191), (300, 2048), (3, 32000), (2, 50257),
          (1, 131072), (5, 131073), (1, 262145), (700, 96), (160, 9000)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,V", SHAPES)
def test_forward_and_gradient(N, V, dt):
    top = (0, 1, 5, 20, 32)[(N + V) % 5]
    scale = (1.0, 0.7, 1.25)[(N + V) % 3]
    z, tokens = make(N, V, dt, seed=N + V, banned=0.1 if N % 2 else 0.0, ignore=-100)
    if V % 2 == 0:
        tokens = tokens.int()
    with_ent = (N + V) % 4 != 1
    out = nl.token_logprobs(z, tokens, scale, top=top, ignore_index=-100, entropy=with_ent)
    torch.cuda.synchronize()
    check(z, tokens, scale, out, top, -100, with_ent)
    dlp, dent, dlse = grads_in(N, V)
    if not with_ent:
        dent = None
    if N % 3 == 0:
        dlse = None
    got = nl.token_logprobs_grad(dlp, z, tokens, out[3], out[1], dent, dlse, scale, ignore_index=-100)
    torch.cuda.synchronize()
    check_grad(z, tokens, scale, got, out[3], out[1], dlp, dent, dlse, -100)


@pytest.mark.parametrize("N,V,top", [(2, 18000, 0), (3, 70000, 0), (44, 70000, 0), (60, 70000, 0), (90, 70001, 0), (130, 70000, 0), (100, 9000, 0),
                                     (170, 9001, 0), (250, 9000, 0), (12, 140000, 20), (30, 140000, 5), (60, 70000, 20), (90, 70000, 3),
                                     (120, 70001, 32), (130, 40000, 20), (200, 40000, 20), (260, 40000, 20), (310, 9000, 20)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_shared_in_every_way(N, V, top, dt):
    """By two, four and eight CTAs, two to four of them an SM, as the number of rows has it."""
    V = V // 2 + 1 if dt == "f32" else V
    z, tokens = make(N, V, dt, seed=N + V, banned=0.05, ignore=-100)
    z[N // 2, : V - 3] = -INF
    out = nl.token_logprobs(z, tokens, top=top, ignore_index=-100)
    check(z, tokens, 1.0, out, top, -100)
    for a, b in zip(nl.token_logprobs(z, tokens, top=top, ignore_index=-100), out):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("dt", list(DT))
def test_each_gradient_alone(dt):
    z, tokens = make(9, 3001, dt, seed=1)
    out = nl.token_logprobs(z, tokens)
    d = grads_in(9, 2)
    for keep in ((0,), (1,), (2,), (0, 1), (1, 2)):
        dlp, dent, dlse = (t if i in keep else None for i, t in enumerate(d))
        got = nl.token_logprobs_grad(dlp, z, tokens if dlp is not None else None, out[3], out[1] if dent is not None else None,
                                     dent, dlse)
        check_grad(z, tokens, 1.0, got, out[3], out[1], dlp, dent, dlse)


def test_leading_dims_and_strides():
    whole = rnd((4, 6, 1100), 3, torch.bfloat16, std=2.0)
    tokens = torch.arange(24, device=DEV).view(4, 6) * 40
    for z in (whole, whole[..., :1001], whole[..., 3:1004], whole[:, :, 16:1000]):
        out = nl.token_logprobs(z, tokens, top=7)
        assert out[0].shape == (4, 6) and out[3].shape == (4, 6, 2) and out[5].shape == (4, 6, 7)
        check(z, tokens, 1.0, out, 7)
        d = [t.view(4, 6) for t in grads_in(24, 4)]
        fresh = nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2])
        check_grad(z, tokens, 1.0, fresh, out[3], out[1], *d)
        # into a tensor of other strides, whose margins stay
        base = torch.full((4, 6, 1200), 5.0, device=DEV, dtype=torch.bfloat16)
        for lo in (16, 17):
            base.fill_(5.0)
            into = base[..., lo:lo + z.shape[-1]]
            nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2], out=into)
            assert torch.equal(into, fresh)
            assert bool((base[..., :lo] == 5.0).all()) and bool((base[..., lo + z.shape[-1]:] == 5.0).all())
        # in place
        mine = whole.clone()
        view = mine.as_strided(z.shape, z.stride(), z.storage_offset())
        nl.token_logprobs_grad(d[0], view, tokens, out[3], out[1], d[1], d[2], out=view)
        assert torch.equal(view, fresh)
        keep = torch.ones_like(mine, dtype=torch.bool)
        keep.as_strided(z.shape, z.stride(), z.storage_offset()).fill_(False)
        assert torch.equal(mine[keep], whole[keep])


def sequences(B, T, V, dt, seed):
    z = rnd((B, T, V), seed, DT[dt], std=2.0)
    return z, torch.tensor(np.random.default_rng(seed).integers(0, V, (B, T)), device=DEV)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("B,T,V", [(3, 9, 1001), (2, 2, 40000), (5, 33, 64)])
def test_each_tokens_logits_with_the_next_token(B, T, V, dt):
    """logits[:, :-1] and tokens[:, 1:], which no one stride reaches: the log probabilities, and the gradient into a fresh
    tensor, into a part of another and in place."""
    whole, tokens = sequences(B, T, V, dt, 40)
    tokens[0, 1], tokens[-1, -1] = -100, -100
    z, t = whole[:, :-1], tokens[:, 1:]
    n = B * (T - 1)
    d = [g.view(B, T - 1) for g in grads_in(n, 41)]
    out = nl.token_logprobs(z, t, 0.9, top=5, ignore_index=-100)
    assert out[0].shape == (B, T - 1) and out[3].shape == (B, T - 1, 2) and out[5].shape == (B, T - 1, 5)
    check(z, t, 0.9, out, 5, -100)
    check(z, t, 0.9, nl.token_logprobs(z, t.int().contiguous(), 0.9, ignore_index=-100), 0, -100)
    check(z.contiguous(), t, 0.9, nl.token_logprobs(z.contiguous(), t, 0.9, ignore_index=-100), 0, -100)
    check(z, None, 0.9, nl.token_logprobs(z, None, 0.9, entropy=False), 0, None, False)
    args = (z, t, out[3], out[1], d[1], d[2], 0.9)
    fresh = nl.token_logprobs_grad(d[0], *args, ignore_index=-100)
    assert fresh.is_contiguous() and fresh.shape == z.shape
    check_grad(z, t, 0.9, fresh, out[3], out[1], *d, -100)
    base = torch.full((B, T + 1, V + 3), 5.0, device=DEV, dtype=DT[dt])
    into = base[:, 1:-1, 2:-1]
    nl.token_logprobs_grad(d[0], *args, ignore_index=-100, out=into)
    assert torch.equal(into, fresh)
    into.fill_(5.0)
    assert bool((base == 5.0).all())
    last = whole[:, -1].clone()
    nl.token_logprobs_grad(d[0], *args, ignore_index=-100, out=z)
    assert torch.equal(z, fresh) and torch.equal(whole[:, -1], last)


def test_rows_of_other_orders_and_shared_ones():
    whole, tokens = sequences(4, 6, 777, "bf16", 42)
    for z, t in ((whole.transpose(0, 1), tokens.t().contiguous()), (whole[::2, 1:4], tokens[::2, 1:4]),
                 (whole[:1].expand(4, 6, 777), tokens), (whole.view(2, 2, 6, 777)[:, :, ::3], tokens.view(2, 2, 6)[:, :, ::3].contiguous())):
        out = nl.token_logprobs(z, t, top=3)
        check(z, t, 1.0, out, 3)
        d = [g.view(t.shape) for g in grads_in(t.numel(), 43)]
        got = nl.token_logprobs_grad(d[0], z, t, out[3], out[1], d[1], d[2])
        check_grad(z, t, 1.0, got, out[3], out[1], *d)


def test_runs_of_rows_captured_and_replayed():
    whole, tokens = sequences(3, 7, 1001, "bf16", 45)
    other, more = sequences(3, 7, 1001, "bf16", 46)
    d = [g.view(3, 6) for g in grads_in(18, 47)]

    def both(whole, tokens):
        z, t = whole[:, :-1], tokens[:, 1:]
        out = nl.token_logprobs(z, t, top=4)
        return [*out, nl.token_logprobs_grad(d[0], z, t, out[3], out[1], d[1], d[2])]

    want = both(other, more)
    both(whole, tokens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(whole, tokens)
    whole.copy_(other)
    tokens.copy_(more)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_runs_of_rows_bad_tokens_and_refusals():
    whole, tokens = sequences(3, 5, 300, "f32", 44)
    z, t = whole[:, :-1], tokens[:, 1:]
    t[2, 1] = 300
    _lib.device_errors()
    out = nl.token_logprobs(z, t)
    torch.cuda.synchronize()
    assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN and out[0][2, 1] == 0
    check(z, t, 1.0, out)
    one = torch.ones(3, 4, device=DEV)
    before, stats = whole.clone(), out[3]

    def bad(err, z, t, out, stats=stats, n=3):
        with pytest.raises(err):
            nl.token_logprobs_grad(one[:n], z, t[:n], stats[:n], out=out)
        assert torch.equal(whole, before)

    bad(nl.NormError, whole[:-1, :-1], t, whole[1:, :-1], n=2)          # the next sequence's logits
    bad(nl.NormError, whole[:1, :-1].expand(3, 4, 300), t, whole[:1, :-1].expand(3, 4, 300))
    bad(nl.NormError, z, t, torch.empty(1, 4, 300, device=DEV).expand(3, 4, 300))
    bad(nl.NormError, z, t, whole[:, 1:])
    bad(nl.NormError, z, t, torch.empty(9000, device=DEV).as_strided((3, 4, 300), (600, 300, 1)))
    bad(ValueError, z, t, torch.empty(3, 4, 299, device=DEV))
    bad(ValueError, z, tokens[:, ::2], None)
    room = torch.zeros(3, 5, 300, device=DEV)                           # statistics inside the gradient's second sequence
    room[1, 0, :24] = stats.flatten()
    bad(nl.NormError, z, t, room[:, :-1], room[1, 0, :24].view(3, 4, 2))
    with pytest.raises(ValueError):
        nl.token_logprobs(z, t[:, :3])
    with pytest.raises(ValueError):
        nl.token_logprobs(z, tokens.t()[1:])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_masked_rows(V, dt):
    """Rows that a mask leaves nothing, one or few tokens, with -inf or the lowest value."""
    low = torch.finfo(DT[dt]).min
    z, tokens = make(10, V, dt, seed=V)
    z[0] = -INF                                 # nothing is left
    z[1] = low                                  # uniform
    z[2] = -INF
    z[2, V - 1] = 1.0                           # one token
    z[3] = low
    z[3, 17] = 0.5
    z[4] = -INF
    z[4, 3], z[4, V // 2] = 2.0, 2.0            # two alike
    z[5, :V // 2] = -INF
    z[6] = 0.0                                  # constant
    z[7] = -INF
    z[7, 5] = low                               # one, of the lowest value
    z[8, V // 2:] = -10000.0
    tokens[2], tokens[3], tokens[4], tokens[7] = V - 1, 17, 0, 5
    for top in (0, 6):
        out = nl.token_logprobs(z, tokens, top=top)
        torch.cuda.synchronize()
        check(z, tokens, 1.0, out, top)
    assert float(out[0][0]) == -INF and float(out[1][0]) == 0.0 and float(out[2][0]) == -INF
    assert abs(float(out[1][1]) - np.log(V)) < 1e-5 and float(out[0][2]) == 0.0 and float(out[1][2]) == 0.0
    assert out[5][0].tolist() == [-1] * 6 and out[5][2].tolist() == [V - 1] + [-1] * 5
    assert out[5][4].tolist() == [3, V // 2] + [-1] * 4 and out[5][6].tolist() == list(range(6))
    d = grads_in(10, 5)
    got = nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2])
    check_grad(z, tokens, 1.0, got, out[3], out[1], *d)
    assert not got[0].any()


@pytest.mark.parametrize("dt", list(DT))
def test_values_that_are_not_finite_stay_in_their_rows(dt):
    z, tokens = make(8, 3000, dt, seed=6)
    good = nl.token_logprobs(z, tokens, top=3)
    d = grads_in(8, 7)
    dgood = nl.token_logprobs_grad(d[0], z, tokens, good[3], good[1], d[1], d[2])
    bad = z.clone()
    bad[1, 77], bad[3, 2999], bad[5] = float("nan"), INF, float("nan")
    out = nl.token_logprobs(bad, tokens, top=3)
    got = nl.token_logprobs_grad(d[0], bad, tokens, out[3], out[1], d[1], d[2])
    rows = torch.tensor([0, 2, 4, 6, 7], device=DEV)
    for a, b in zip(out, good):
        assert torch.equal(a[rows], b[rows])
    assert torch.equal(got[rows], dgood[rows])
    for r in (1, 3, 5):
        for t in out[:3]:
            assert bool(t[r].isnan())
        assert bool(got[r].isnan().all())
    assert out[5][1].tolist() == O.top_ids(n64(bad[1:2]), 3)[0].tolist()
    assert int(out[5][3, 0]) == 2999 and out[5][5].tolist() == [-1, -1, -1] and float(out[3][3, 0]) == INF


@pytest.mark.parametrize("top", [1, 5, 20, 32])
@pytest.mark.parametrize("dt", list(DT))
def test_alternatives_of_many_kinds_of_rows(dt, top):
    """Ascending, descending and constant rows, ties, plateaus, and the largest logits crowded into few threads' chunks."""
    V = 20011
    r = np.random.default_rng(8)
    rows = [np.arange(V) / 64.0, -np.arange(V) / 64.0, np.zeros(V), r.integers(0, 3, V) * 1.0, r.integers(0, 200, V) / 8.0,
            np.where(np.arange(V) % 4096 < 32, 50 + r.random(V), r.random(V)),   # columns of few threads
            np.where(np.arange(V) < 4000, 7.0, r.random(V)), np.where(np.arange(V) >= V - 4000, 7.0, r.random(V)),
            -np.abs(r.normal(size=V)) * 1e-3, np.where(np.arange(V) % 2 == 0, -0.0, 0.0), r.normal(size=V)]
    z = torch.tensor(np.stack(rows)).to(DT[dt]).to(DEV)
    check(z, None, 1.0, nl.token_logprobs(z, top=top), top)
    # one row at a time, shared by a cluster
    for i in range(z.shape[0]):
        check(z[i:i + 1], None, 1.0, nl.token_logprobs(z[i:i + 1], top=top), top)


@pytest.mark.parametrize("dt", list(DT))
def test_more_candidates_than_fit(dt):
    """Thousands of the largest logits in the chunks of a dozen threads: they are found one after another."""
    GE = 32 // torch.finfo(DT[dt]).bits * 8
    V = 512 * GE * 32
    z = rnd((400, V), 9, DT[dt])  # many rows: one CTA a row, 512 threads
    chunk = torch.arange(V, device=DEV) // GE % 512
    z[:, (chunk >= 36) & (chunk < 48)] += 100.0
    for top in (20, 32):
        out = nl.token_logprobs(z, top=top)
        check(z[:3], None, 1.0, tuple(None if t is None else t[:3] for t in out), top)
        assert torch.equal(out[5], torch.sort(z.float(), dim=1, descending=True, stable=True)[1][:, :top])


@pytest.mark.parametrize("dt", list(DT))
def test_more_candidates_than_fit_in_some_parts_of_a_row(dt):
    """Rows shared by clusters of eight CTAs of 1536 chunks: in two of the CTAs the largest logits are in the chunks of a dozen
    of the 256 threads, which find them one after another, in the others they are not."""
    GE = 32 // torch.finfo(DT[dt]).bits * 8
    part = 256 * 6
    V = 8 * part * GE
    z = rnd((3, V), 9, DT[dt])
    chunk = torch.arange(V, device=DEV) // GE
    few = (chunk % 256 >= 36) & (chunk % 256 < 48)
    z[:, few & ((chunk // part == 1) | (chunk // part == 6))] += 60.0
    z[1, chunk // part == 3] += 50.0
    z[2] = torch.where(few, 9.0, z[2])  # equal ones, in all of them
    for top in (20, 32):
        out = nl.token_logprobs(z, top=top)
        check(z, None, 1.0, out, top)


def test_more_alternatives_than_tokens():
    z = rnd((3, 4), 10, torch.float32)
    out = nl.token_logprobs(z, top=9)
    check(z, None, 1.0, out, 9)
    assert out[5][:, 4:].eq(-1).all() and out[4][:, 4:].eq(-INF).all()


def test_tokens_outside_the_vocabulary():
    z, tokens = make(6, 300, "f32", seed=11)
    tokens[1], tokens[2], tokens[4] = -1, 300, 1 << 40
    _lib.device_errors()
    out = nl.token_logprobs(z, tokens)
    torch.cuda.synchronize()
    assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
    check(z, tokens, 1.0, out)
    assert out[0][1] == out[0][2] == out[0][4] == 0
    d = grads_in(6, 12)
    got = nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2])
    torch.cuda.synchronize()
    assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
    check_grad(z, tokens, 1.0, got, out[3], out[1], *d)
    # an ignored one is no error, wherever it lies
    out = nl.token_logprobs(z[:2], tokens[:2], ignore_index=-1)
    torch.cuda.synchronize()
    assert _lib.device_errors() == 0 and out[0][1] == 0


def test_the_least_token_is_no_ignored_one():
    """Without ignore_index every token outside the vocabulary is an error, the least of its type too."""
    z, tokens = make(5, 300, "f32", seed=23)
    d = grads_in(5, 24)
    for t in (tokens, tokens.int()):
        t[2] = torch.iinfo(t.dtype).min
        _lib.device_errors()
        out = nl.token_logprobs(z, t)
        torch.cuda.synchronize()
        assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
        check(z, t, 1.0, out)
        got = nl.token_logprobs_grad(d[0], z, t, out[3], out[1], d[1], d[2])
        torch.cuda.synchronize()
        assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
        check_grad(z, t, 1.0, got, out[3], out[1], *d)
        nl.token_logprobs(z, t, ignore_index=int(torch.iinfo(torch.int32).min))
        torch.cuda.synchronize()
        assert _lib.device_errors() == (_lib.NORM_DEVICE_ERR_BAD_TOKEN if t.dtype == torch.long else 0)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 30.0, 1e4])
def test_scales(scale):
    z, tokens = make(5, 4001, "f32", seed=13)
    out = nl.token_logprobs(z, tokens, scale, top=3)
    check(z, tokens, scale, out, 3)
    d = grads_in(5, 14)
    got = nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2], scale)
    check_grad(z, tokens, scale, got, out[3], out[1], *d)


@pytest.mark.parametrize("std", [1e-3, 30.0, 1000.0])
def test_logits_near_together_and_far_apart(std):
    z, tokens = make(5, 9001, "f32", seed=15, std=std)
    out = nl.token_logprobs(z, tokens, top=3)
    check(z, tokens, 1.0, out, 3)
    d = grads_in(5, 16)
    check_grad(z, tokens, 1.0, nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2]), out[3], out[1], *d)
    # ascending: every chunk has a new maximum
    z = z.sort(1)[0]
    check(z, tokens, 1.0, nl.token_logprobs(z, tokens), 0)


def test_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    N, V = 17000, 131072
    assert N * V > 2 ** 31
    one, tokens = make(1, V, "bf16", seed=17)
    z = one.expand(N, V).contiguous()
    tokens = tokens.expand(N).contiguous()
    out = nl.token_logprobs(z, tokens, top=2)
    check(z[:1], tokens[:1], 1.0, tuple(t[:1] for t in out), 2)
    for t in out:
        assert bool((t == t[:1]).all())
    d = [t.expand(N).contiguous() for t in grads_in(1, 18)]
    got = nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2], out=z)
    check_grad(one, tokens[:1], 1.0, got[:1], out[3][:1], out[1][:1], *(t[:1] for t in d))
    assert bool((got == got[:1]).all())


def test_outputs_of_many_rows_keep_nothing_else():
    """A kept log probability must not hold the alternatives of all rows."""
    z, tokens = make(3000, 64, "bf16", seed=25)
    out = nl.token_logprobs(z, tokens, top=32)
    assert sum(t.numel() * t.element_size() for t in out) > 1 << 20
    for t in out:
        assert t.untyped_storage().nbytes() == t.numel() * t.element_size() and t.storage_offset() == 0
    check(z, tokens, 1.0, out, 32)


def test_repeated_calls_have_the_same_bits():
    z, tokens = make(37, 50001, "bf16", seed=19)
    first = nl.token_logprobs(z, tokens, top=20)
    for _ in range(3):
        for a, b in zip(nl.token_logprobs(z, tokens, top=20), first):
            assert torch.equal(a, b)


def test_capture_replay_and_two_streams():
    z, tokens = make(6, 40001, "bf16", seed=20)
    z2, t2 = make(6, 40001, "bf16", seed=21)
    d = grads_in(6, 22)

    def both(z, tokens):
        out = nl.token_logprobs(z, tokens, top=4)
        return [*out, nl.token_logprobs_grad(d[0], z, tokens, out[3], out[1], d[1], d[2])]

    want, want2 = both(z, tokens), both(z2, t2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    zg, tg = z.clone(), tokens.clone()
    with torch.cuda.graph(graph):
        got = both(zg, tg)
    for src, tok, w in ((z2, t2, want2), (z, tokens, want)):
        zg.copy_(src)
        tg.copy_(tok)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    res = [None, None]
    for _ in range(4):
        for i, a in enumerate(((z, tokens), (z2, t2))):
            with torch.cuda.stream(streams[i]):
                res[i] = both(*a)
    torch.cuda.synchronize()
    for r, w in zip(res, (want, want2)):
        for a, b in zip(r, w):
            assert torch.equal(a, b)


def test_one_row_without_a_batch_dim_and_inference_mode():
    z, tokens = make(1, 777, "bf16", seed=30)
    want = nl.token_logprobs(z, tokens, top=3)
    got = nl.token_logprobs(z[0], tokens[0], top=3)
    assert got[0].shape == () and got[3].shape == (2,) and got[5].shape == (3,)
    with torch.inference_mode():
        more = nl.token_logprobs(z, tokens.view(1), top=3)
        one = torch.ones((), device=DEV)
        d = nl.token_logprobs_grad(one, z[0], tokens[0], got[3], got[1], one)
    for a, b, c in zip(got, want, more):
        assert torch.equal(a.reshape(b.shape), b) and torch.equal(b, c)
    assert d.shape == (777,)
    check_grad(z, tokens, 1.0, d.view(1, -1), want[3], want[1], one.view(1), one.view(1), None)
    got = nl.token_logprobs(z.requires_grad_(), tokens, top=3)
    assert not got[0].requires_grad
    got[0].fill_(7.0)  # ordinary tensors, whatever they share
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a, b)


def test_empty_batch():
    z = torch.empty(0, 30, device=DEV)
    out = nl.token_logprobs(z, torch.empty(0, device=DEV, dtype=torch.long), top=2)
    assert [t.numel() for t in out] == [0] * 6
    e = torch.empty(0, device=DEV)
    assert nl.token_logprobs_grad(e, z, torch.empty(0, device=DEV, dtype=torch.long), out[3], out[1], e, e).shape == (0, 30)


def test_binding_refusals():
    z, tokens = make(4, 100, "bf16")
    out = nl.token_logprobs(z, tokens)
    d = grads_in(4, 1)

    def bad(err, *a, **kw):
        with pytest.raises(err):
            nl.token_logprobs(*a, **kw)

    bad(TypeError, z.double(), tokens)
    bad(ValueError, z[:, ::2], tokens)
    bad(ValueError, z, tokens[:3])
    bad(ValueError, z, tokens.cpu())
    bad(TypeError, z, tokens.float())
    bad(ValueError, z, torch.stack([tokens, tokens], 1)[:, 0])
    bad(ValueError, z, tokens, top=33)
    bad(ValueError, z, tokens, top=-1)
    bad(nl.NormError, z, tokens, 0.0)
    bad(nl.NormError, z, tokens, -1.0)
    bad(nl.NormError, z, tokens, float("nan"))
    bad(nl.NormError, z[:1].expand(4, 100), tokens)
    g = nl.token_logprobs_grad
    for a, kw in (((d[0], z, None, out[3]), {}), ((None, z, tokens, out[3]), {}), ((d[0], z, tokens, out[3], None, d[1]), {}),
                  ((d[0][:3], z, tokens, out[3]), {}), ((d[0].bfloat16(), z, tokens, out[3]), {}),
                  ((d[0].sum().expand(4), z, tokens, out[3]), {}), ((d[0], z, tokens, out[3][:, :1]), {}),
                  ((d[0], z, tokens, out[3].cpu()), {}), ((d[0], z, tokens, out[3]), dict(out=z[:3])),
                  ((d[0], z, tokens, out[3]), dict(out=torch.empty(4, 100, device=DEV)))):
        with pytest.raises(ValueError):
            g(*a, **kw)
    with pytest.raises(nl.NormError):
        g(d[0], z, tokens, out[3], out=torch.empty(1, 100, device=DEV, dtype=torch.bfloat16).expand(4, 100))
    with pytest.raises(nl.NormError):
        g(d[0], z, tokens, out[3], scale=0.0)
    with pytest.raises(nl.NormError):
        g(d[0][:3], z[:3], tokens[:3], out[3][:3], out=z[1:])


def test_together_as_a_model_uses_them():
    """Tokens -> embedding -> one attention block with normed, rotated heads -> join -> logits -> log probabilities, and
    the way back to every parameter, against autograd in 64 bits (the products and the softmax are torch's).

    fp32 throughout: sums of at most 512 terms, a handful of layers: relative to each gradient's largest element
    1e-4, four orders above U and three below a term left out."""
    B, T, C, Hq, Hk, D, V, eps = 2, 24, 64, 4, 2, 16, 500, 1e-5
    f = torch.float32
    p = {n: rnd(s, i + 30, f, m, std) for i, (n, s, m, std) in enumerate([
        ("table", (V, C), 0.0, 1.0), ("g0", (C,), 1.0, 0.1), ("wq", (C, Hq * D), 0.0, 0.2), ("wk", (C, Hk * D), 0.0, 0.2),
        ("wv", (C, Hk * D), 0.0, 0.2), ("wo", (Hq * D, C), 0.0, 0.2), ("gq", (D,), 1.0, 0.1), ("gk", (D,), 1.0, 0.1),
        ("gpost", (C,), 1.0, 0.1), ("gate", (C,), 0.7, 0.1), ("gpre", (C,), 1.0, 0.1)])}
    r = np.random.default_rng(1)
    tokens = torch.tensor(r.integers(0, V, (B, T)), device=DEV)
    targets = torch.tensor(r.integers(0, V, (B, T)), device=DEV)
    targets[0, :3] = -100
    a = torch.arange(T, device=DEV, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    cos, sin = a.cos().float(), a.sin().float()
    wlp, went, wlse = (rnd((B, T), 50 + i, f, std=s) for i, s in enumerate((1.0, 0.2, 0.1)))
    mask = torch.ones(T, T, device=DEV, dtype=torch.bool).tril()

    def attend(q, k, v):
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
        s = (q @ k.transpose(-1, -2) * D ** -0.5).masked_fill(~mask, -INF).softmax(-1)
        return (s @ v).transpose(1, 2).reshape(B, T, Hq * D)

    # here
    y0, h0, r0 = nl.embedding_rms(tokens, p["table"], p["g0"], eps, 2.0)
    q, k, v = (y0 @ p["wq"]).unflatten(-1, (Hq, D)), (y0 @ p["wk"]).unflatten(-1, (Hk, D)), (y0 @ p["wv"]).unflatten(-1, (Hk, D))
    qr, kr = nl.head_rms_rotary(q, k, p["gq"], p["gk"], cos, sin, None, eps)
    leaves = [t.detach().requires_grad_() for t in (qr, kr, v)]
    o = attend(*leaves)
    x = o.detach() @ p["wo"]
    y, h, rp, rn = nl.sandwich_rms(x, h0, p["gpost"], p["gate"], p["gpre"], eps, residual_scale=0.9)
    logits = y @ p["table"].t()
    lp, ent, lse, stats, tl, ti = nl.token_logprobs(logits, targets, 0.8, top=3, ignore_index=-100)
    dz = nl.token_logprobs_grad(wlp, logits, targets, stats, ent, went, wlse, 0.8, ignore_index=-100)
    g = {}
    dy = dz @ p["table"]
    dx, dh, g["gpost"], g["gate"], g["gpre"] = nl.sandwich_rms_grad(dy, x, h, rp, rn, p["gpost"], p["gate"], p["gpre"],
                                                                    residual_scale=0.9)
    g["wo"] = o.detach().flatten(0, 1).t() @ dx.flatten(0, 1)
    dqr, dkr, dv = torch.autograd.grad(o, leaves, dx @ p["wo"].t())
    dq, dk, g["gq"], g["gk"] = nl.head_rms_rotary_grad(dqr, dkr, q, k, p["gq"], p["gk"], cos, sin, None, eps)
    dy0 = torch.zeros_like(y0)
    for n, d in (("wq", dq), ("wk", dk), ("wv", dv)):
        d = d.reshape(B, T, -1)
        g[n] = y0.flatten(0, 1).t() @ d.flatten(0, 1)
        dy0 += d @ p[n].t()
    dh0, _, g["g0"] = nl.fused_add_rms_backward(dy0, h0, r0, p["g0"], dh, residual_grad="none")
    g["table"] = nl.embedding_grad(dh0, tokens, V, 2.0) + dz.flatten(0, 1).t() @ y.flatten(0, 1)

    # autograd, 64 bits
    P = {n: t.double().requires_grad_() for n, t in p.items()}

    def rms(x, w):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w

    def turn(x):
        c, s = cos.double()[:, None], sin.double()[:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    h0 = P["table"][tokens] * 2.0
    y0 = rms(h0, P["g0"])
    q, k, v = ((y0 @ P[n]).unflatten(-1, (H, D)) for n, H in (("wq", Hq), ("wk", Hk), ("wv", Hk)))
    x = attend(turn(rms(q, P["gq"])), turn(rms(k, P["gk"])), v) @ P["wo"]
    y = rms(0.9 * h0 + P["gate"] * rms(x, P["gpost"]), P["gpre"])
    logp = torch.log_softmax(y @ P["table"].t() * 0.8, -1)
    rlse = torch.logsumexp(y @ P["table"].t() * 0.8, -1)
    rent = -(logp.exp() * logp).sum(-1)
    rlp = torch.where(targets < 0, 0.0, logp.gather(-1, targets.clamp(min=0)[..., None])[..., 0])
    want = torch.autograd.grad((rlp * wlp).sum() + (rent * went).sum() + (rlse * wlse).sum(), list(P.values()))
    # Besides what is relative: a token far ahead of the others makes the sum of exponentials 1 + d with d next to
    # nothing, of which fp32 keeps U at best, and log(1 + d) with it: the 200 U (+ 8 U E|x|, E|x| < 1 there) above are
    # absolute, and the entropies here (1e-6 at most) are smaller than that.
    for a, b in ((lp, rlp), (ent, rent), (lse, rlse)):
        b = b.detach()
        assert float((a - b).abs().max()) < 1e-4 * float(b.abs().max()) + 208 * U
    assert torch.equal(ti, logp.topk(3, -1).indices)
    for (n, _), w in zip(P.items(), want):
        assert g[n].shape == w.shape and float((g[n] - w).abs().max()) < 1e-4 * float(w.abs().max()), n


def test_zz_no_device_errors():
    torch.cuda.synchronize()
    assert _lib.device_errors() == 0

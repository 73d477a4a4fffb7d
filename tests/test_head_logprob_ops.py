"""The per-head norm with rotation and the log probabilities on the CPU: the
oracle against torch autograd in 64 bits and difference quotients, and the C
ABI's and the binding's refusals (fake addresses; every call is rejected, or has
no rows, before it reaches the GPU)."""

import ctypes

import numpy as np
import pytest
import torch

import rmsnorm_ln_fwd_gb300 as nl
from oracle import head_oracle as O
from rmsnorm_ln_fwd_gb300 import _build, _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2
I32, I64 = 0, 1
M = 0x1000000  # fake, well-separated addresses: M, 2*M, ...


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


# ------------------------------------------------------------------ the oracle

def _angles(N, R, seed):
    p = np.random.default_rng(seed).integers(0, 50, N)
    a = p[:, None] * 100.0 ** (-np.arange(R // 2) / max(1, R // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(8, 8), (10, 6), (7, 2), (5, 0)])
def test_head_oracle_is_autograd(D, R, interleaved):
    r = np.random.default_rng(D + R)
    N, H, eps = 5, 3, 1e-5
    x, dy, g = r.normal(size=(N, H, D)), r.normal(size=(N, H, D)), r.normal(1, 0.2, D)
    cos, sin = _angles(N, R, 1) if R else (None, None)
    tx, tg = torch.tensor(x, requires_grad=True), torch.tensor(g, requires_grad=True)
    n = torch.nn.functional.rms_norm(tx, (D,), tg, eps)
    y = n
    if R:
        # as a product of complex numbers
        h = n[..., :R]
        z = torch.complex(h[..., 0::2], h[..., 1::2]) if interleaved else torch.complex(h[..., :R // 2], h[..., R // 2:])
        z = z * torch.complex(torch.tensor(cos), torch.tensor(sin))[:, None]
        t = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
        y = torch.cat([t, n[..., R:]], -1)
    (y * torch.tensor(dy)).sum().backward()
    assert np.allclose(O.head_forward(x, g, cos, sin, eps, interleaved), y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dg = O.head_backward(dy, x, g, cos, sin, eps, interleaved)
    assert np.allclose(dx, tx.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(dg, tg.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_head_oracle_is_the_difference_quotient():
    r = np.random.default_rng(0)
    N, H, D, R, eps, step = 2, 2, 6, 4, 1e-5, 1e-6
    x, dy, g = r.normal(size=(N, H, D)), r.normal(size=(N, H, D)), r.normal(1, 0.2, D)
    cos, sin = _angles(N, R, 1)
    dx, dg = O.head_backward(dy, x, g, cos, sin, eps)

    def loss(x, g):
        return (O.head_forward(x, g, cos, sin, eps) * dy).sum()

    # the quotient's own error: third derivatives of order 10 times step^2, rounding 1e-15 / step
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += step
        down[i] -= step
        assert abs((loss(up, g) - loss(down, g)) / (2 * step) - dx[i]) < 1e-7
    for i in range(D):
        up, down = g.copy(), g.copy()
        up[i] += step
        down[i] -= step
        assert abs((loss(x, up) - loss(x, down)) / (2 * step) - dg[i]) < 1e-7


def test_logprob_oracle_is_autograd():
    r = np.random.default_rng(2)
    N, V, a = 6, 11, 1.3
    z, tokens = r.normal(0, 2, (N, V)), np.array([0, 3, 10, -100, 5, 42])
    z[1, 4:] = -np.inf
    z[4, 5] = -np.inf
    dlp, dh, dl = r.normal(size=(3, N))
    logprob, entropy, lse, m, l, x, p = O.logprob_forward(z, tokens, a, ignore=-100)
    t = torch.tensor(z, requires_grad=True)
    lp = torch.log_softmax(t * a, 1)
    ent = -(lp.exp() * lp.masked_fill(lp == -np.inf, 0.0)).sum(1)
    tl = torch.logsumexp(t * a, 1)
    has = torch.tensor([True, True, True, False, True, False])
    at = torch.tensor(tokens).where(has, torch.tensor(0))
    tlp = torch.where(has, lp.gather(1, at[:, None])[:, 0], torch.tensor(0.0, dtype=torch.float64))
    for got, want in ((logprob, tlp), (entropy, ent), (lse, tl)):
        assert np.allclose(got, want.detach().numpy(), rtol=1e-12, atol=1e-12)
    use = torch.tensor([True, True, True, True, False, True])  # the log probability of an impossible token is -inf
    ((tlp * torch.tensor(dlp))[use].sum() + (ent * torch.tensor(dh)).sum() + (tl * torch.tensor(dl)).sum()).backward()
    d = np.where(use.numpy(), dlp, 0.0)
    got = O.logprob_backward(d, z, tokens, m, l, entropy, dh, dl, a, ignore=-100)
    assert np.allclose(got, t.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_logprob_oracle_is_the_difference_quotient():
    r = np.random.default_rng(3)
    N, V, a, step = 3, 5, 0.7, 1e-6
    z, tokens = r.normal(0, 2, (N, V)), np.array([0, 3, 4])
    dlp, dh, dl = r.normal(size=(3, N))
    _, entropy, _, m, l, _, _ = O.logprob_forward(z, tokens, a)
    got = O.logprob_backward(dlp, z, tokens, m, l, entropy, dh, dl, a)

    def loss(z):
        lp, h, lse, *_ = O.logprob_forward(z, tokens, a)
        return (lp * dlp + h * dh + lse * dl).sum()

    for i in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[i] += step
        down[i] -= step
        assert abs((loss(up) - loss(down)) / (2 * step) - got[i]) < 1e-7


def test_logprob_oracle_edges():
    z = np.full((4, 3), -np.inf)
    z[1] = -3e38
    z[2, 1] = 0.0
    z[3] = [1.0, 1.0, np.nan]
    logprob, entropy, lse, *_ = O.logprob_forward(z[:3], np.array([0, 1, 1]), 1.0)
    assert np.array_equal(logprob, [-np.inf, -np.log(3), 0.0]) and np.allclose(entropy, [0.0, np.log(3), 0.0])
    assert lse[0] == -np.inf and lse[2] == 0.0
    assert np.array_equal(O.top_ids(z, 2), [[-1, -1], [0, 1], [1, -1], [0, 1]])
    assert np.array_equal(O.top_ids(z[1:2], 5), [[0, 1, 2, -1, -1]])


# ------------------------------------------------------------------ refusals of the C ABI

def _heads(p, sb=0, st=0, sh=0):
    return ctypes.byref(_lib.Heads(p, sb, st, sh)) if p is not None else None


def _rotation(**kw):
    a = dict(cos=8 * M, cos_stride=32, sin=9 * M, sin_stride=32, rows=100, columns=64, dtype=F32, interleaved=0,
             positions=None, position_type=I64, position_batch_stride=0, position_token_stride=0)
    a.update(kw)
    return ctypes.byref(_lib.Rotation(**a))


# (B, T, heads, D) = (2, 3, 4, 64) contiguous
S = dict(sb=3 * 4 * 64, st=4 * 64, sh=64)


def _rotary(lib, **kw):
    a = dict(q=_heads(M, **S), hq=4, k=_heads(2 * M, **S), hk=4, gq=None, gk=None, qo=_heads(3 * M, **S),
             ko=_heads(4 * M, **S), rot=_rotation(), B=2, T=3, D=64, eps=1e-6, xd=BF16, wd=BF16)
    a.update(kw)
    return lib.head_rms_rotary(a["q"], a["hq"], a["k"], a["hk"], a["gq"], a["gk"], a["qo"], a["ko"], a["rot"], a["B"],
                               a["T"], a["D"], a["eps"], a["xd"], a["wd"], None)


def test_rotary_refusals(lib):
    nan = float("nan")
    for name, kw in dict(
            eps0=dict(eps=0.0), epsnan=dict(eps=nan), D0=dict(D=0), wide=dict(D=513), B=dict(B=-1), T=dict(T=-1),
            noheads=dict(hq=0, hk=0), negative=dict(hq=-1), many=dict(hq=65536), nullq=dict(q=None), nullk=dict(k=None),
            nulldata=dict(q=_heads(0, **S)), nullout=dict(qo=None), odd=dict(q=_heads(M + 1, **S)),
            oddout=dict(ko=_heads(4 * M + 1, **S)), oddgamma=dict(gq=5 * M + 1),
            stride=dict(q=_heads(M, -1, 256, 64)), far=dict(q=_heads(M, 1 << 62, 256, 64)),
            # outputs whose heads share elements
            expanded=dict(qo=_heads(3 * M, S["sb"], S["st"], 0)), tight=dict(qo=_heads(3 * M, S["sb"], S["st"], 63)),
            short=dict(qo=_heads(3 * M, S["sb"], 255, 64)),
            # outputs over inputs or each other
            qoverk=dict(qo=_heads(2 * M, **S)), shifted=dict(qo=_heads(M + 2, **S)),
            restrided=dict(qo=_heads(M, S["sb"], S["st"] * 2, 64)), both=dict(ko=_heads(3 * M, **S)),
            halfway=dict(ko=_heads(3 * M + 128 * 5, **S)), params=dict(gq=3 * M), paramk=dict(gk=4 * M + 64),
            table=dict(rot=_rotation(cos=3 * M)), positions=dict(rot=_rotation(positions=3 * M + 8)),
            # the rotation
            R0=dict(rot=_rotation(columns=0)), odd_columns=dict(rot=_rotation(columns=63)),
            past=dict(rot=_rotation(columns=66)),
            # 33 units of 16 columns
            units=dict(D=512, rot=_rotation(columns=510, cos_stride=255, sin_stride=255), q=_heads(M, 6144, 2048, 512),
                       k=_heads(2 * M, 6144, 2048, 512), qo=_heads(3 * M, 6144, 2048, 512), ko=_heads(4 * M, 6144, 2048, 512)),
            tokens=dict(B=1, T=1 << 31, rot=None), rows0=dict(rot=_rotation(rows=0)), rows=dict(rot=_rotation(rows=2)),
            negrows=dict(rot=_rotation(rows=-1)), cosstride=dict(rot=_rotation(cos_stride=31)), nocos=dict(rot=_rotation(cos=None)),
            nosin=dict(rot=_rotation(sin=None)), oddcos=dict(rot=_rotation(cos=8 * M + 2)),
            oddpos=dict(rot=_rotation(positions=10 * M + 4)),
            negpos=dict(rot=_rotation(positions=10 * M, position_token_stride=-1)),
            # what belongs to heads that are not there
            gammak=dict(hk=0, k=None, ko=None, gk=5 * M)).items():
        assert _rotary(lib, **kw) == INVALID, name
    assert _rotary(lib, xd=7) == UNSUPPORTED
    assert _rotary(lib, xd=F32, wd=BF16) == UNSUPPORTED
    assert _rotary(lib, rot=_rotation(dtype=F16)) == UNSUPPORTED
    assert _rotary(lib, rot=_rotation(positions=10 * M, position_type=9)) == UNSUPPORTED
    assert _rotary(lib, T=0, q=None, k=None, qo=None, ko=None) == OK
    assert _rotary(lib, B=0, rot=None) == OK


def test_rotary_fused_parts_that_touch_are_refused(lib):
    # queries and keys of one projection, (B, T, (4 + 2 + 2) * 64), in place or as parts of another buffer
    row = 8 * 64
    f = dict(sb=3 * row, st=row, sh=64)
    q, k = _heads(M, **f), _heads(M + 4 * 64 * 2, **f)
    ok = dict(q=q, k=k, hk=2)
    for name, kw in dict(
            k_over_q=dict(qo=q, ko=_heads(M + 3 * 64 * 2, **f)),      # the last query head
            q_over_k=dict(qo=_heads(M + 64 * 2, **f), ko=k),
            wraps=dict(qo=q, ko=_heads(M + 7 * 64 * 2, **f)),         # the second key head is the next token's first
            outs=dict(qo=_heads(3 * M, **f), ko=_heads(3 * M + 2 * (4 * 64 - 8), **f)),
            other_period=dict(qo=q, ko=_heads(M + 4 * 64 * 2, 3 * row, row + 64, 64))).items():
        assert _rotary(lib, **{**ok, **kw}) == INVALID, name


def _rgrad(lib, **kw):
    a = dict(dyq=_heads(5 * M, **S), q=_heads(M, **S), hq=4, dyk=_heads(6 * M, **S), k=_heads(2 * M, **S), hk=4, gq=None,
             gk=None, dq=_heads(3 * M, **S), dk=_heads(4 * M, **S), dgq=11 * M, dgk=12 * M, rot=_rotation(), ws=13 * M,
             wsb=1 << 20, B=2, T=3, D=64, eps=1e-6, xd=BF16, wd=BF16)
    a.update(kw)
    return lib.head_rms_rotary_grad(a["dyq"], a["q"], a["hq"], a["dyk"], a["k"], a["hk"], a["gq"], a["gk"], a["dq"],
                                    a["dk"], a["dgq"], a["dgk"], a["rot"], a["ws"], a["wsb"], a["B"], a["T"], a["D"],
                                    a["eps"], a["xd"], a["wd"], None)


def test_rotary_grad_refusals(lib):
    for name, kw in dict(
            eps=dict(eps=-1.0), D=dict(D=600), nully=dict(dyq=None), nullx=dict(k=None), nulldx=dict(dq=None),
            over_x=dict(dq=_heads(M, **S)), over_other_dy=dict(dq=_heads(6 * M, **S)), shifted=dict(dq=_heads(5 * M + 2, **S)),
            both=dict(dk=_heads(3 * M, **S)), expanded=dict(dk=_heads(4 * M, S["sb"], 0, 64)), dgammas=dict(dgq=12 * M + 2),
            dgamma_odd=dict(dgk=12 * M + 1), dgamma_x=dict(dgq=M + 64), dgamma_dx=dict(dgk=3 * M), dgamma_gamma=dict(gq=11 * M),
            gamma_dx=dict(gk=4 * M), rows=dict(rot=_rotation(rows=2)), dgamma_cos=dict(dgq=8 * M),
            nokeys=dict(hk=0, dyk=None, k=None, dk=None)).items():
        assert _rgrad(lib, **kw) == INVALID, name
    for name, kw in dict(none=dict(ws=None), odd=dict(ws=13 * M + 8), over=dict(ws=5 * M), under=dict(ws=11 * M - 64)).items():
        assert _rgrad(lib, **kw) == WORKSPACE, name
    assert _rgrad(lib, xd=F16, wd=BF16) == UNSUPPORTED
    assert _rgrad(lib, T=0, dgq=None, dgk=None) == OK


def test_parts_of_heads_side_by_side(lib):
    # (B, T, heads, 3, D): a head's query, key and value beside one another; ws=None shows that all else is accepted
    f = dict(sb=3 * 4 * 192, st=4 * 192, sh=192)

    def parts(p):
        return _heads(p, **f), _heads(p + 2 * 64, **f)

    def ask(**kw):
        x, dy, dx = parts(M), parts(5 * M), parts(3 * M)
        a = dict(q=x[0], k=x[1], dyq=dy[0], dyk=dy[1], dq=dx[0], dk=dx[1], ws=None)
        return _rgrad(lib, **{**a, **kw})

    assert ask() == WORKSPACE
    dy = parts(5 * M)
    assert ask(dq=dy[0], dk=dy[1]) == WORKSPACE  # in place
    assert ask(dk=_heads(3 * M + 2 * 128, **f)) == WORKSPACE
    assert ask(hk=1, dk=_heads(3 * M + 2 * 128, f["sb"], f["st"], 0)) == WORKSPACE  # one key head beside the first query's
    # (B, T, 4 + 4 heads) with room behind each sequence that is no multiple of a token's
    g = dict(sb=3 * 512 + 24, st=512, sh=64)
    assert ask(dq=_heads(3 * M, **g), dk=_heads(3 * M + 2 * 256, **g)) == WORKSPACE
    assert ask(dq=_heads(3 * M, **g), dk=_heads(3 * M + 2 * 255, **g)) == INVALID
    for name, kw in dict(
            early=dict(dk=_heads(3 * M + 2 * 63, **f)), late=dict(dk=_heads(3 * M + 2 * 129, **f)),
            crossed=dict(dq=dy[1], dk=dy[0]), halfway=dict(dk=_heads(3 * M + 2 * 64 + 1, **f)),
            other_period=dict(dk=_heads(3 * M + 2 * 64, f["sb"], f["st"], 128)),
            other_tokens=dict(dk=_heads(3 * M + 2 * 64, f["sb"] + 64, f["st"], 192))).items():
        assert ask(**kw) == INVALID, name


def test_parts_are_taken_only_where_no_element_is_shared(lib):
    """Gradients of queries and keys in one buffer, in random layouts, against the elements that they have; ws=None shows that
    all else is accepted."""
    r = np.random.default_rng(5)
    taken = 0
    for _ in range(20000):
        B, T, hq, hk, D = (int(v) for v in (*r.integers(1, 4, 2), *r.integers(1, 4, 2), r.choice([1, 2, 4])))

        def layout(heads):
            sizes = {"sb": B, "st": T, "sh": heads}
            at, out = int(r.choice([D, D, 2 * D, 3 * D, D + 1])), {}
            for name in r.permutation(["sb", "st", "sh"]):
                out[name] = at
                at = at * sizes[name] + int(r.choice([0, 0, 0, D, 1]))
            return out

        fq = layout(max(hq, hk) if r.random() < 0.5 else hq + hk)
        fk = fq if r.random() < 0.7 else layout(hk)
        off = int(r.integers(0, 1 + max(fq.values())) if r.random() < 0.3 else r.integers(0, 8) * D)

        def elements(f, heads, at):
            i = np.indices((B, T, heads, D)).reshape(4, -1)
            return set((i[0] * f["sb"] + i[1] * f["st"] + i[2] * f["sh"] + i[3] + at).tolist())

        eq, ek = elements(fq, hq, 0), elements(fk, hk, off)
        if len(eq) < B * T * hq * D or len(ek) < B * T * hk * D:
            continue
        got = _rgrad(lib, hq=hq, hk=hk, B=B, T=T, D=D, rot=None, xd=F32, wd=F32, ws=None, dq=_heads(3 * M, **fq),
                     dk=_heads(3 * M + 4 * off, **fk))
        assert got in (INVALID, WORKSPACE)
        assert got == INVALID or not eq & ek, (B, T, hq, hk, D, fq, fk, off)
        taken += got == WORKSPACE
    assert taken > 3000


def _lp(lib, **kw):
    a = dict(z=M, ld=64, tok=2 * M, it=I64, scale=1.0, ignore=-100, lp=3 * M, ent=4 * M, lse=5 * M, st=6 * M, tlp=7 * M,
             tid=8 * M, top=5, N=4, V=64, dt=BF16)
    a.update(kw)
    return lib.token_logprobs(a["z"], a["ld"], a["tok"], a["it"], a["scale"], a["ignore"], a["lp"], a["ent"], a["lse"],
                              a["st"], a["tlp"], a["tid"], a["top"], a["N"], a["V"], a["dt"], None)


def test_logprob_refusals(lib):
    inf, nan = float("inf"), float("nan")
    for kw in (dict(z=None), dict(z=M + 1), dict(ld=63), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25), dict(N=-1),
               dict(N=(1 << 28) + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan), dict(scale=3e38),
               dict(top=-1), dict(top=33), dict(top=0), dict(tlp=None), dict(tid=None), dict(tok=None), dict(lp=None),
               dict(tok=2 * M + 4), dict(lp=3 * M + 2), dict(st=6 * M + 4), dict(tid=8 * M + 4), dict(lp=M), dict(ent=2 * M),
               dict(lse=4 * M), dict(st=4 * M + 8), dict(tid=7 * M), dict(ent=8 * M + 64),
               dict(tok=None, lp=None, ent=None, lse=None, st=None, top=0, tlp=None, tid=None)):
        assert _lp(lib, **kw) == INVALID, kw
    assert _lp(lib, dt=5) == UNSUPPORTED
    assert _lp(lib, it=3) == UNSUPPORTED
    assert _lp(lib, N=0, z=None, tok=None, lp=None) == OK


def _lpg(lib, **kw):
    a = dict(dlp=M, z=2 * M, ld=64, tok=3 * M, it=I32, st=4 * M, ent=5 * M, dent=6 * M, dlse=7 * M, scale=1.0, ignore=-1,
             dz=8 * M, lddz=64, N=4, V=64, dt=F16)
    a.update(kw)
    return lib.token_logprobs_grad(a["dlp"], a["z"], a["ld"], a["tok"], a["it"], a["st"], a["ent"], a["dent"], a["dlse"],
                                   a["scale"], a["ignore"], a["dz"], a["lddz"], a["N"], a["V"], a["dt"], None)


def test_logprob_grad_refusals(lib):
    for kw in (dict(z=None), dict(st=None), dict(dz=None), dict(tok=None), dict(ent=None), dict(dlp=None, dent=None, dlse=None),
               dict(ld=63), dict(lddz=10), dict(dz=2 * M + 2), dict(dz=2 * M, lddz=65), dict(dz=M), dict(dz=3 * M),
               dict(dz=4 * M + 8), dict(dz=5 * M), dict(dz=6 * M), dict(dz=7 * M), dict(st=4 * M + 4), dict(dlp=M + 2),
               dict(scale=0.0), dict(scale=float("nan")), dict(V=0), dict(N=-2)):
        assert _lpg(lib, **kw) == INVALID, kw
    assert _lpg(lib, dt=9) == UNSUPPORTED
    assert _lpg(lib, it=9) == UNSUPPORTED
    assert _lpg(lib, N=0, z=None) == OK


# ------------------------------------------------------------------ the binding

def test_heads_view_of_strided_tensors(lib):
    view = _lib.bind().heads_view
    t = torch.empty(2, 5, 8 * 16)
    q = t[..., :64].unflatten(-1, (4, 16))
    assert view(q) == (2, 5, 4, 16, 640, 128, 16)
    assert view(q.transpose(1, 2).contiguous().transpose(1, 2)) == (2, 5, 4, 16, 320, 16, 80)
    assert view(q[0]) == (1, 5, 4, 16, 0, 128, 16)
    for bad in (q[..., ::2], q[0, 0], q[None]):
        with pytest.raises(ValueError):
            view(bad)


def test_runs_of_rows_and_their_tokens(lib):
    """Rows that no single stride reaches, and tokens of a slice, as runs (first row, first token), rows a run and row stride."""
    runs = _lib.bind().token_runs
    z, t = torch.empty(3, 5, 7), torch.arange(15).view(3, 5)
    assert runs(z, None, None) == (15, 7, [(0, 0, 0)])
    assert runs(z, t, None) == (15, 7, [(0, 0, 0)])
    assert runs(z[:, :-1], t[:, 1:], None) == (4, 7, [(0, 0, 0), (35, 5, 0), (70, 10, 0)])  # tokens from their own first one
    assert runs(z[:, :-1], t[:, 1:].reshape(-1), None) == (4, 7, [(0, 0, 0), (35, 4, 0), (70, 8, 0)])
    assert runs(z[:, :-1], t[:, 1:].contiguous(), None) == (4, 7, [(0, 0, 0), (35, 4, 0), (70, 8, 0)])
    assert runs(z[:, :4].contiguous(), t[:, 1:], None) == (4, 7, [(0, 0, 0), (28, 5, 0), (56, 10, 0)])
    assert runs(z[:, :1], t[:, :1].contiguous(), None) == (3, 35, [(0, 0, 0)])
    assert runs(z[:, :1], t[:, 1:2], None) == (1, 7, [(0, 0, 0), (35, 5, 0), (70, 10, 0)])  # a token of each sequence
    assert runs(z.transpose(0, 1), t.t().contiguous(), None) == (3, 35, [(7 * i, 3 * i, 0) for i in range(5)])
    assert runs(z, t, torch.empty(3, 9, 8)[:, 2:7, 1:]) == (5, 7, [(0, 0, 0), (35, 5, 72), (70, 10, 144)])
    w = torch.empty(2, 3, 5, 7)
    assert runs(w[:, :, 1:], None, None) == (4, 7, [(35 * i, 4 * i, 0) for i in range(6)])
    assert runs(w[:, :2], None, None) == (10, 7, [(0, 0, 0), (105, 10, 0)])
    assert runs(w[:, :0], torch.empty(2, 0, 5, dtype=torch.long), None)[0] == 0
    assert runs(z[0, 0], t[0, 0], None) == (1, 7, [(0, 0, 0)])
    assert runs(z[:1].expand(3, 5, 7), t, None) == (5, 7, [(0, 0, 0), (0, 5, 0), (0, 10, 0)])
    for tokens in (t.t(), t[:, ::2], t[:2, 1:]):  # of other dims than the rows', or no neighbours
        with pytest.raises(ValueError):
            runs(z, tokens, None)


def test_host_tensors_are_refused(lib):
    x, c = torch.zeros(3, 2, 8), torch.zeros(4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        nl.head_rms_rotary(x, x, cos=c, sin=c)
    with pytest.raises(ValueError, match="CUDA"):
        nl.head_rms_rotary_grad(x, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        nl.token_logprobs(torch.zeros(3, 8), torch.zeros(3, dtype=torch.long))
    with pytest.raises(ValueError, match="CUDA"):
        nl.token_logprobs_grad(None, torch.zeros(3, 8), None, torch.zeros(3, 2))


def test_columns_of_a_head_that_is_partly_rotated_in_halves(lib):
    for D in (1, 2, 63, 64, 495, 496, 497, 500, 511, 512, 513):
        for R in range(2, D + 1, 2):
            for pairs in (0, 1):
                ok = D <= 512 and (pairs or -(-R // 16) + -(-(D - R) // 16) <= 32)
                assert ok or D > 496
                got = _rotary(lib, D=D, T=0, rot=_rotation(columns=R, cos_stride=R // 2, sin_stride=R // 2, interleaved=pairs))
                assert got == (OK if ok else INVALID), (D, R, pairs)


def test_workspace_size_needs_a_width(lib):
    assert lib.head_rms_rotary_workspace_bytes(0, 0) == 0
    assert lib.head_rms_rotary_workspace_bytes(513, 0) == 0

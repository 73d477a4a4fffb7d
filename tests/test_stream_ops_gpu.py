"""The residual-stream operators on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (U = 2^-24, half an fp32 step; S the sum of the
magnitudes of the terms an element is formed from):

* a row sum of H terms: at most 16 or H/256 serial additions in a thread (the
  widest shape of each kernel family) and 20 tree levels, two roundings a term
  before it: K = H/256 + 40 steps of U relative to the sum of magnitudes.  A
  reciprocal norm halves that and adds rsqrtf's two steps.
* an element of y: K*U on its terms and the norm's error.  dx combines two row
  sums, the second formed from the first: 2K.
* a sum over rows: each term's error, N/64 serial additions (units are never
  fewer than 64 for these N; 32 in a tile) and 20 tree levels.
* a value stored in fewer bits: half a step, finfo.eps/2 of the value (and half
  the smallest subnormal), on top.
"""

import numpy as np
import pytest
import torch

import rmsnorm_ln_fwd_gb300 as nl
from normtest import Guarded
from oracle import stream_oracle as S
from rmsnorm_ln_fwd_gb300 import _lib, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_ln_fwd_gb300 import _build
    _build.build()
    _lib.device_errors()


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def steps(H):
    return H / 256 + 40


def close(got, ref, slack, what):
    """|got - ref| <= slack + half a step of got's type (fp32 itself: U)."""
    dt = got.dtype
    half = U if dt == torch.float32 else torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    g = n64(got).reshape(np.shape(ref))
    err = np.abs(g - ref)
    tol = slack + half * (np.abs(ref) + slack) + tiny
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    if not np.all(err <= tol):
        i = np.unravel_index(np.argmax(err - tol), err.shape)
        raise AssertionError(f"{what}: {int((err > tol).sum())} of {err.size} beyond the bound; at {i} got {g[i]!r} "
                             f"want {ref[i]!r} (bound {np.broadcast_to(tol, err.shape)[i]:.3g})")


def rnd(shape, seed, dt, mean=0.0, std=1.0, roles=("x",)):
    return synth.normal(shape, seed, roles[0], mean=mean, std=std, dtype=dt).to(DEV)


def join_inputs(N, H, dt, wdt, gates, seed=0, gdt=None):
    g = None
    if gates:
        g = rnd((H,) if gates == 1 else (gates, H), seed + 5, gdt or wdt, 0.5, 0.5)
    return dict(x=rnd((N, H), seed, dt), res=rnd((N, H), seed + 1, dt, std=2.0), gpost=rnd((H,), seed + 2, wdt, 1.0, 0.1),
                gpre=rnd((H,), seed + 3, wdt, 1.0, 0.1), gate=g, dy=rnd((N, H), seed + 6, dt),
                dh=rnd((N, H), seed + 7, dt, std=0.5))


def check_join(c, out, eps, alpha, post, pre):
    y, h, rpost, rpre = out
    x, res, gpost, gate, gpre = (n64(c[k]) for k in ("x", "res", "gpost", "gate", "gpre"))
    N, H = x.shape
    k = steps(H) * U
    ry, rh, rrpost, rrpre = S.sandwich_forward(x, res, gpost if post else None, gate, gpre if pre else None, eps,
                                               alpha, post, pre)
    terms = np.abs(alpha * res) + np.abs(rh - alpha * res)
    close(h, rh, k * terms, "h")
    if post:
        close(rpost, rrpost, k * rrpost, "rstd_post")
    if pre:
        # sum h^2 moves by at most 2 |h| . dh: relative to it, the rms of the terms over that of h
        spread = np.sqrt((terms ** 2).mean(1)) * rrpre
        close(rpre, rrpre, k * (1 + spread) * rrpre, "rstd_pre")
        close(y, ry, k * (terms * rrpre[:, None] * np.abs(gpre) + np.abs(ry) * (1 + spread[:, None])), "y")
    else:
        assert y is None and rpre is None


SHAPES = [(1, 1), (1, 4096), (2, 7), (5, 1000), (33, 1001), (64, 256), (18, 2056), (40, 5120), (6, 10240), (4, 16384),
          (3, 16390), (2, 40008), (700, 512), (310, 48), (2500, 128), (9, 24)]


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,H", SHAPES)
def test_join(N, H, dt, post, pre):
    eps, alpha = 1e-5, 0.75
    gates = {0: 0, 1: 1}.get((N + H) % 3, 1 if N == 1 else next(b for b in (5, 3, 2, 11, 7, N) if N % b == 0))
    wdt = DT["f32"] if H % 2 else DT[dt]
    c = join_inputs(N, H, DT[dt], wdt, gates, seed=N + H)
    out = nl.sandwich_rms(c["x"], c["res"], c["gpost"] if post else None, c["gate"], c["gpre"] if pre else None, eps,
                          residual_scale=alpha, post_norm=post, pre_norm=pre)
    torch.cuda.synchronize()
    check_join(c, out, eps, alpha, post, pre)


def check_join_grad(c, out, rpost, rpre, alpha, N_serial=None):
    dx, dres, dgpost, dgate, dgpre = out
    x, h, gpost, gate, gpre, dy, dh = (n64(c[k]) for k in ("x", "res", "gpost", "gate", "gpre", "dy", "dh"))
    N, H = x.shape
    post, pre = rpost is not None, rpre is not None
    rpo, rpr = n64(rpost), n64(rpre)
    ref = S.sandwich_backward(dy if pre else None, x, h if pre else None, rpo, rpr, gpost if post else None, gate,
                              gpre if pre else None, dh, alpha)
    k = steps(H) * U
    # magnitudes of the terms
    sdh = np.abs(dh)
    hh = np.zeros_like(x)
    if pre:
        hh = np.abs(h * rpr[:, None])
        g = np.abs(dy * gpre)
        C = (g * hh).mean(1, keepdims=True)
        sdh = sdh + rpr[:, None] * (g + hh * C)
    rows = S._rows_of_gate(gate, N, H)
    w, oh, ro = np.abs(rows), np.abs(x), 1.0
    if post:
        ro = rpo[:, None]
        oh = oh * ro
        w = w * np.abs(gpost)
    sk = (w * oh * sdh).mean(1, keepdims=True) if post else 0.0
    close(dres, ref[1], 2 * k * np.abs(alpha) * sdh, "dres")
    close(dx, ref[0], 2 * k * ro * (w * sdh + oh * sk), "dx")
    kr = 2 * k + (N / 64 + 20) * U
    if post:
        close(dgpost, ref[2], kr * (np.abs(rows) * sdh * oh).sum(0), "dgamma_post")
    else:
        assert dgpost is None
    if gate is not None:
        B = gate.reshape(-1, H).shape[0]
        terms = (sdh * oh * (np.abs(gpost) if post else 1.0)).reshape(B, N // B, H).sum(1).reshape(gate.shape)
        close(dgate, ref[3], kr * terms, "dgate")
    else:
        assert dgate is None
    if pre:
        close(dgpre, ref[4], kr * (np.abs(dy) * hh).sum(0), "dgamma_pre")
    else:
        assert dgpre is None


def run_join_grad(c, post, pre, alpha=0.75, eps=1e-5, **kw):
    """The gradient at the stream given by c["res"] (as the stored h)."""
    rpost = torch.from_numpy(S._rstd(n64(c["x"]), eps)).float().to(DEV) if post else None
    rpre = torch.from_numpy(S._rstd(n64(c["res"]), eps)).float().to(DEV) if pre else None
    out = nl.sandwich_rms_grad(c["dy"] if pre else None, c["x"], c["res"] if pre else None, rpost, rpre,
                               c["gpost"] if post else None, c["gate"], c["gpre"] if pre else None, c["dh"],
                               residual_scale=alpha, **kw)
    torch.cuda.synchronize()
    return out, rpost, rpre


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,H", SHAPES)
def test_join_grad(N, H, dt, post, pre):
    gates = {0: 0, 1: 1}.get((N + H) % 3, 1 if N == 1 else next(b for b in (5, 3, 2, 11, 7, N) if N % b == 0))
    wdt = DT["f32"] if H % 2 else DT[dt]
    c = join_inputs(N, H, DT[dt], wdt, gates, seed=N + H)
    out, rpost, rpre = run_join_grad(c, post, pre)
    check_join_grad(c, out, rpost, rpre, 0.75)


@pytest.mark.parametrize("N,B", [(2000, 2), (2000, 8), (2000, 400), (2000, 1000), (2000, 2000), (1333, 43), (1333, 31),
                                 (608, 304), (303, 3)])
@pytest.mark.parametrize("H,dt", [(256, "bf16"), (1024, "f16"), (2048, "bf16"), (130, "f32"), (1024, "f32")])
def test_join_gates_of_runs(N, B, H, dt):
    """Runs that end inside a unit, cross units, are longer and shorter than a
    unit, and of one row."""
    c = join_inputs(N, H, DT[dt], torch.float32, B, seed=B)
    out = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], 1e-5, residual_scale=0.75)
    check_join(c, out, 1e-5, 0.75, True, True)
    out, rpost, rpre = run_join_grad(c, True, True)
    check_join_grad(c, out, rpost, rpre, 0.75)


def padded(t, ld, off=0):
    """A copy of t in rows `ld` apart, `off` elements into a larger buffer whose
    every other element is a sentinel; returns (view, buffer, mask of the rest)."""
    N, H = t.shape
    buf = torch.full((off + N * ld + 8,), -77.0, dtype=t.dtype, device=t.device)
    view = buf[off:off + N * ld].view(N, ld)[:, :H]
    view.copy_(t)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[off:off + N * ld].view(N, ld)[:, :H] = False
    return view, buf, rest


@pytest.mark.parametrize("N,H,ld,off", [(37, 1024, 1032, 8), (37, 1024, 1024, 1), (21, 1000, 1003, 3), (5, 5120, 5136, 16),
                                        (300, 64, 65, 0), (3, 16384, 16400, 0)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_join_strides_and_margins(N, H, ld, off, dt):
    """Padded and shifted rows give the contiguous call's bits or stay within the
    bound, and what lies between and behind the rows is left as it was."""
    c = join_inputs(N, H, DT[dt], DT[dt], 1, seed=H)
    p = {k: padded(c[k], ld, off)[0] for k in ("x", "res", "dy", "dh")}
    bufs = {k: padded(torch.zeros_like(c["x"]), ld, off) for k in ("y", "h", "dx", "dr")}
    # a gate that is a column slice of a wider tensor
    wide = torch.full((1, 2 * H + 64), 5.0, dtype=DT[dt], device=DEV)
    wide[:, H:2 * H] = c["gate"]
    gate = wide[:, H:2 * H]
    y, h, rpost, rpre = nl.sandwich_rms(p["x"], p["res"], c["gpost"], gate, c["gpre"], 1e-5, residual_scale=0.75,
                                        h_out=bufs["h"][0], out=bufs["y"][0])
    check_join(c, (y, h, rpost, rpre), 1e-5, 0.75, True, True)
    cc = {**c, "gate": gate}
    rp = torch.from_numpy(S._rstd(n64(c["x"]), 1e-5)).float().to(DEV)
    rq = torch.from_numpy(S._rstd(n64(c["res"]), 1e-5)).float().to(DEV)
    out = nl.sandwich_rms_grad(p["dy"], p["x"], p["res"], rp, rq, c["gpost"], gate, c["gpre"], p["dh"],
                               residual_scale=0.75, dx=bufs["dx"][0], dres=bufs["dr"][0])
    torch.cuda.synchronize()
    assert out[3].shape == gate.shape
    check_join_grad(cc, out, rp, rq, 0.75)
    for k, (view, buf, rest) in bufs.items():
        assert torch.all(buf[rest] == -77.0), k


@pytest.mark.parametrize("N,H,dt", [(50, 1024, "bf16"), (7, 1001, "f16"), (20, 5120, "bf16"), (4, 16384, "f32"),
                                    (2, 70000, "bf16")])
def test_join_in_place(N, H, dt):
    c = join_inputs(N, H, DT[dt], DT[dt], 1, seed=1)
    ref = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], residual_scale=0.5)
    for name in ("x", "res"):
        d = {k: None if v is None else v.clone() for k, v in c.items()}
        y, h, a, b = nl.sandwich_rms(d["x"], d["res"], d["gpost"], d["gate"], d["gpre"], residual_scale=0.5,
                                     h_out=d[name])
        assert h is d[name]
        for got, want in zip((y, h, a, b), ref):
            assert torch.equal(got, want)
    want, rpost, rpre = run_join_grad(c, True, True)
    d = {k: None if v is None else v.clone() for k, v in c.items()}
    got = nl.sandwich_rms_grad(d["dy"], d["x"], d["res"], rpost, rpre, d["gpost"], d["gate"], d["gpre"], d["dh"],
                               residual_scale=0.75, dx=d["dy"], dres=d["dh"])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_join_guards_and_bits():
    """Margins of every output survive, and a second call gives the same bits."""
    N, H, B = 400, 1040, 5
    c = join_inputs(N, H, torch.bfloat16, torch.bfloat16, B, seed=4)
    rp = torch.from_numpy(S._rstd(n64(c["x"]), 1e-5)).float().to(DEV)
    rq = torch.from_numpy(S._rstd(n64(c["res"]), 1e-5)).float().to(DEV)
    first = None
    for _ in range(3):
        g = [Guarded((N, H), torch.bfloat16, DEV) for _ in range(4)]
        y, h, a, b = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], out=g[0].t, h_out=g[1].t)
        out = nl.sandwich_rms_grad(c["dy"], c["x"], c["res"], rp, rq, c["gpost"], c["gate"], c["gpre"], c["dh"],
                                   dx=g[2].t, dres=g[3].t)
        torch.cuda.synchronize()
        assert all(x.ok() for x in g)
        now = [t.clone() for t in (y, h, a, b, *out)]
        if first is None:
            first = now
        assert all(torch.equal(p, q) for p, q in zip(first, now))


def test_join_skips_what_is_not_asked():
    c = join_inputs(30, 256, torch.bfloat16, torch.bfloat16, 3, seed=4)
    out, rp, rq = run_join_grad(c, True, True)
    bare, _, _ = run_join_grad(c, True, True, need_param_grads=False)
    assert torch.equal(out[0], bare[0]) and torch.equal(out[1], bare[1])
    assert bare[2] is None and bare[3] is None and bare[4] is None
    y, h, a, b = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], save_stats=False)
    assert a is None and b is None


def test_join_no_rows():
    x = torch.empty((0, 64), device=DEV, dtype=torch.bfloat16)
    r = torch.empty(0, device=DEV)
    gate = torch.ones((4, 64), device=DEV, dtype=torch.bfloat16)
    y, h, a, b = nl.sandwich_rms(x, x, None, gate)
    assert y.shape == h.shape == (0, 64)
    dx, dr, dp, dg, dn = nl.sandwich_rms_grad(x, x, x, r, r, None, gate, None, None)
    assert not dp.any() and not dg.any() and not dn.any() and dg.shape == (4, 64)


@pytest.mark.parametrize("H", [64, 1001, 5120, 16384])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_join_bad_rows_stay_alone(H, bad):
    """A row with a NaN or an infinity leaves the other rows' bits as they were."""
    c = join_inputs(9, H, torch.bfloat16, torch.bfloat16, 1, seed=2)
    want = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"])
    x = c["x"].clone()
    x[4, H // 2] = bad
    got = nl.sandwich_rms(x, c["res"], c["gpost"], c["gate"], c["gpre"])
    keep = [i for i in range(9) if i != 4]
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(got[0][4]).all()


@pytest.mark.parametrize("H", [64, 1001, 5120])
def test_join_grad_without_post_norm_leaves_x_out_of_dx(H):
    """dx = gate * dh then: an infinite x reaches dgate, not dx."""
    c = join_inputs(6, H, torch.bfloat16, torch.bfloat16, 1, seed=2)
    want, _, _ = run_join_grad(c, False, True)
    c["x"] = c["x"].clone()
    c["x"][3, H // 3] = float("inf")
    got, _, _ = run_join_grad(c, False, True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[4], want[4])
    assert not torch.isfinite(got[3][H // 3]) and torch.isfinite(got[3][:H // 3]).all()


def test_join_cancelling_stream():
    """A block output that cancels the stream almost everywhere: the second
    norm's sum is far smaller than its terms.  The rows are exact multiples, so
    the bound is that of the terms."""
    N, H = 16, 2048
    x = rnd((N, H), 3, torch.float32)
    x = torch.sign(x)  # rstd of x is 1 up to eps
    res = -x.clone()
    res[:, 5] += 0.01
    c = dict(x=x, res=res, gpost=torch.ones(H, device=DEV), gate=None, gpre=torch.ones(H, device=DEV))
    out = nl.sandwich_rms(x, res, c["gpost"], None, c["gpre"], 1e-6)
    check_join(c, out, 1e-6, 1.0, True, True)


def test_join_zero_rows():
    """Rows of zeros: the norms give eps^-1/2 and zeros, no NaN."""
    x = torch.zeros((4, 512), device=DEV, dtype=torch.bfloat16)
    y, h, a, b = nl.sandwich_rms(x, x, eps=1e-4)
    assert not y.any() and not h.any() and torch.allclose(a, torch.full_like(a, 100.0)) and torch.equal(a, b)


# ------------------------------------------------------------------ lookup

@pytest.mark.parametrize("it", [torch.int32, torch.int64])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,H,V", [(1, 1, 1), (1, 4096, 50), (8, 1000, 7), (33, 1001, 100), (700, 512, 2000), (18, 2056, 9),
                                   (40, 5120, 30), (5, 16384, 6), (3, 16390, 4), (2, 40008, 3), (1000, 64, 500)])
def test_lookup(N, H, V, dt, it):
    table = rnd((V, H), H, DT[dt])
    gamma = rnd((H,), 2, DT["f32"] if H % 2 else DT[dt], 1.0, 0.1)
    tokens = torch.from_numpy(np.random.default_rng(N).integers(0, V, N)).to(DEV, it)
    y, h, rstd = nl.embedding_rms(tokens, table, gamma, 1e-5, 1.5)
    only = nl.embedding_lookup(tokens, table, 1.5)
    torch.cuda.synchronize()
    assert torch.equal(only, h) and _lib.device_errors() == 0
    ry, rh, rr = S.lookup_forward(tokens.tolist(), n64(table), 1.5, n64(gamma), 1e-5)
    k = steps(H) * U
    close(h, rh, U * np.abs(rh), "h")
    close(rstd, rr, k * rr, "rstd")
    close(y, ry, 2 * k * np.abs(ry), "y")


@pytest.mark.parametrize("H", [64, 1001, 2048])
def test_lookup_bad_tokens(H):
    table = rnd((10, H), 1, torch.bfloat16)
    tokens = torch.tensor([3, 10, -1, 9, 2 ** 40, 0], device=DEV)
    y, h, rstd = nl.embedding_rms(tokens, table, None, 1e-4)
    torch.cuda.synchronize()
    assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
    assert not h[[1, 2, 4]].any() and not y[[1, 2, 4]].any()
    assert torch.equal(h[[0, 3, 5]], table[[3, 9, 0]])
    dt = nl.embedding_grad(h, tokens, 10)
    torch.cuda.synchronize()
    assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
    assert torch.equal(dt[[3, 9, 0]], h[[0, 3, 5]]) and not dt[[1, 2, 4, 5, 6, 7, 8]].any()
    nl.embedding_lookup(tokens[:1], table)
    torch.cuda.synchronize()
    assert _lib.device_errors() == 0


def test_lookup_shapes_strides_margins():
    big = rnd((20, 300), 1, torch.float16)
    table = big[:, 3:260]  # padded, misaligned rows
    tokens = torch.arange(12, device=DEV).view(3, 4)
    g = Guarded((3, 4, 257), torch.float16, DEV)
    h = nl.embedding_lookup(tokens, table, 0.5, out=g.t)
    torch.cuda.synchronize()
    assert h.shape == (3, 4, 257) and g.ok()
    assert torch.equal(h.view(12, 257), (table[:12].float() * 0.5).half())
    assert nl.embedding_lookup(tokens[:0], table).shape == (0, 4, 257)
    with pytest.raises(ValueError, match="contiguous"):
        nl.embedding_lookup(tokens.t(), table)
    with pytest.raises(TypeError, match="int32 or int64"):
        nl.embedding_lookup(tokens.float(), table)


KINDS = ["uniform", "skewed", "one", "distinct", "padded", "two"]


def make_tokens(kind, N, V):
    r = np.random.default_rng(N + V)
    if kind == "uniform":
        t = r.integers(0, V, N)
    elif kind == "skewed":
        t = np.clip(np.floor(np.exp(r.random(N) * np.log(V + 1))) - 1, 0, V - 1).astype(np.int64)
    elif kind == "one":
        t = np.full(N, V // 2)
    elif kind == "distinct":
        t = r.permutation(max(N, V))[:N] % V
    elif kind == "two":
        t = np.where(r.random(N) < 0.5, 0, V - 1)
    else:
        t = np.where(r.random(N) < 0.4, V - 1, r.integers(0, V, N))
    return t


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,H,V,dt,odt", [(1, 64, 5, "bf16", "bf16"), (31, 8, 1, "f32", "f32"), (32, 100, 40, "bf16", "f32"),
                                          (33, 1001, 600, "f16", "f16"), (65, 256, 513, "bf16", "bf16"),
                                          (2000, 48, 70000, "bf16", "f32"), (5000, 16, 300000, "f32", "f32"),
                                          (3333, 520, 1000, "f16", "f32"), (300, 4104, 64, "bf16", "bf16"),
                                          (9000, 24, 511, "f32", "f32"), (20000, 8, 5000, "f32", "f32"),
                                          (40000, 16, 140000, "bf16", "f32"), (70000, 8, 300, "f32", "f32"),
                                          (5000, 1040, 3000, "bf16", "bf16"), (4097, 1001, 2500, "f32", "f32")])
def test_lookup_grad(kind, N, H, V, dt, odt):
    tokens = make_tokens(kind, N, V)
    pad = V - 1 if kind == "padded" else -1
    dh = rnd((N, H), N, DT[dt])
    tok = torch.from_numpy(tokens).to(DEV, torch.int32 if N % 2 else torch.int64)
    g = Guarded((V, H), DT[odt], DEV)
    out = nl.embedding_grad(dh, tok, V, 1.5, padding_idx=None if pad < 0 else pad, out=g.t)
    torch.cuda.synchronize()
    assert out is g.t and g.ok() and _lib.device_errors() == 0
    d = n64(dh)
    ref = S.lookup_backward(d, tokens, V, 1.5, pad)
    terms = S.lookup_backward(np.abs(d), tokens, V, 1.5, pad)
    # serial additions: 32 in a tile, the tiles of an id, and its scale
    counts = np.bincount(tokens, minlength=V)[:, None]
    close(out, ref, (40 + counts / 32) * U * terms, "dtable")
    # absent rows are exact zeros, a second call gives the same bits
    keep = out.clone()
    assert not keep[torch.from_numpy((counts[:, 0] == 0) | (np.arange(V) == pad)).to(DEV)].any()
    again = nl.embedding_grad(dh, tok, V, 1.5, padding_idx=None if pad < 0 else pad, param_dtype=DT[odt])
    assert torch.equal(keep, again)
    # accumulated into what is there: only the named rows change, by the same sums
    base = rnd((V, H), 9, DT[odt])
    acc = nl.embedding_grad(dh, tok, V, 1.5, padding_idx=None if pad < 0 else pad, out=base.clone(), accumulate=True)
    torch.cuda.synchronize()
    b = n64(base)
    close(acc, ref + b, (42 + counts / 32) * U * (terms + np.abs(b)), "dtable accumulated")
    absent = torch.from_numpy((counts[:, 0] == 0) | (np.arange(V) == pad)).to(DEV)
    assert torch.equal(acc[absent], base[absent])


def test_lookup_grad_strided_table_and_none():
    N, H, V = 50, 96, 30
    dh = rnd((N, H), 1, torch.bfloat16)
    tok = torch.from_numpy(make_tokens("uniform", N, V)).to(DEV)
    for ld, off in ((104, 8), (99, 1)):
        view, buf, rest = padded(torch.ones((V, H), dtype=torch.bfloat16, device=DEV), ld, off)
        out = nl.embedding_grad(dh, tok, V, out=view)
        torch.cuda.synchronize()
        assert torch.all(buf[rest] == -77.0)
        assert torch.equal(out.contiguous(), nl.embedding_grad(dh, tok, V))
    none = nl.embedding_grad(dh[:0], tok[:0], V)
    assert none.shape == (V, H) and not none.any()
    kept = torch.ones((V, H), device=DEV)
    nl.embedding_grad(dh[:0], tok[:0], V, out=kept, accumulate=True)
    assert torch.all(kept == 1)
    with pytest.raises(ValueError, match="padding_idx"):
        nl.embedding_grad(dh, tok, V, padding_idx=V)
    with pytest.raises(ValueError, match="accumulate"):
        nl.embedding_grad(dh, tok, V, accumulate=True)
    with pytest.raises(ValueError, match="rows for"):
        nl.embedding_grad(dh, tok[:-1], V)


# ------------------------------------------------------------------ together

def test_join_refusals_of_tensors():
    x = torch.zeros((6, 64), device=DEV, dtype=torch.bfloat16)
    r = torch.ones(6, device=DEV)
    v = torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="divide"):
        nl.sandwich_rms(x, x.clone(), gate=torch.ones((4, 64), device=DEV))
    with pytest.raises(ValueError, match="columns"):
        nl.sandwich_rms(x, x.clone(), gate=torch.ones(63, device=DEV))
    with pytest.raises(TypeError, match="gate"):
        nl.sandwich_rms(x, x.clone(), gate=torch.ones(64, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError, match="post_norm"):
        nl.sandwich_rms(x, x.clone(), v, post_norm=False)
    with pytest.raises(nl.NormError):
        nl.sandwich_rms(x, x.clone(), post_norm=False, pre_norm=False)
    with pytest.raises(nl.NormError):
        nl.sandwich_rms(x, x.clone(), out=x)
    with pytest.raises(ValueError, match="come together"):
        nl.sandwich_rms_grad(x, x, None, r, r)
    with pytest.raises(ValueError, match="no norm"):
        nl.sandwich_rms_grad(None, x, None, None, None, dh_in=x)
    with pytest.raises(ValueError, match="no gradient"):
        nl.sandwich_rms_grad(None, x, None, r, None)
    with pytest.raises(nl.NormError):
        nl.sandwich_rms_grad(x, x.clone(), x.clone(), r, r.clone(), workspace=torch.empty(16, device=DEV))
    with pytest.raises(ValueError, match="elements"):
        nl.sandwich_rms_grad(x, x.clone(), x.clone(), r[:5], r)


def _model(tokens, table, params, gates, steps_, dev):
    """Tokens -> stream; blocks (a fixed elementwise map stands for each) joined
    to it; gradients back to the table.  Returns every gradient."""
    y, h, r = nl.embedding_rms(tokens, table, params[0], 1e-5, 1.5)
    saved = []
    for i in range(steps_):
        x = y * (0.5 + i)
        y2, h2, rpost, rpre = nl.sandwich_rms(x, h, params[1 + 2 * i], gates[i], params[2 + 2 * i], 1e-5,
                                              residual_scale=0.9)
        saved.append((x, h2, rpost, rpre))
        y, h = y2, h2
    dy, dh = torch.cos(h), torch.sin(h)
    grads = []
    for i in reversed(range(steps_)):
        x, h2, rpost, rpre = saved[i]
        dx, dh, dpost, dgate, dpre = nl.sandwich_rms_grad(dy, x, h2, rpost, rpre, params[1 + 2 * i], gates[i],
                                                          params[2 + 2 * i], dh, residual_scale=0.9)
        dy = dx * (0.5 + i)
        grads += [dpost, dgate, dpre]
    h0 = nl.embedding_lookup(tokens, table, 1.5)
    dh0, _, dg = nl.fused_add_rms_backward(dy, h0, r, params[0], dh, residual_grad="none")
    return [y, h, *grads, dg, nl.embedding_grad(dh0, tokens, table.shape[0], 1.5)]


def _model_inputs(H=512, V=300, B=4, T=25, dt=torch.float32):
    table = rnd((V, H), 1, dt)
    params = [rnd((H,), 10 + i, dt, 1.0, 0.1) for i in range(5)]
    gates = [rnd((B, 1, H), 20, dt, 0.5, 0.3), rnd((H,), 21, dt, 0.5, 0.3)]
    tokens = torch.from_numpy(make_tokens("skewed", B * T, V)).view(B, T).to(DEV)
    return tokens, table, params, gates


def test_stream_end_to_end_is_autograd():
    """Lookup, two joins and all their gradients in fp32 against torch autograd
    in 64 bits.  Eight operators of at most 2K steps each in a row, each step
    relative to terms a few times the values: 64 K U of the largest value."""
    tokens, table, params, gates = _model_inputs()
    got = _model(tokens, table, params, gates, 2, DEV)
    leaf = [t.double().requires_grad_() for t in [table, *params, *gates]]
    tab, ps, gs = leaf[0], leaf[1:6], leaf[6:]

    def norm(v, g):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * g

    h = 1.5 * tab[tokens]
    y = norm(h, ps[0])
    for i in range(2):
        h = 0.9 * h + gs[i] * norm(y * (0.5 + i), ps[1 + 2 * i])
        y = norm(h, ps[2 + 2 * i])
    torch.autograd.backward([y, h], [torch.cos(got[1]).double(), torch.sin(got[1]).double()])
    want = [y, h, ps[3].grad, gs[1].grad, ps[4].grad, ps[1].grad, gs[0].grad, ps[2].grad, ps[0].grad, tab.grad]
    for i, (a, b) in enumerate(zip(got, want)):
        b = b.detach()
        err = (a.double() - b.view(a.shape)).abs().max().item()
        assert err <= 64 * steps(512) * U * b.abs().max().item(), (i, err)


def test_stream_captured_and_on_other_streams():
    """The whole run captured into two graphs, replayed in turn and on another
    stream, gives the eager call's bits with new inputs too."""
    tokens, table, params, gates = _model_inputs(dt=torch.bfloat16)
    want = _model(tokens, table, params, gates, 2, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _model(tokens, table, params, gates, 2, DEV)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _model(tokens, table, params, gates, 2, DEV)
        graphs.append((g, outs))
    for k in range(2):
        if k:
            tokens.copy_(torch.flip(tokens, [1]))
            table.mul_(0.5)
            want = _model(tokens, table, params, gates, 2, DEV)
        for g, outs in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("N,H,B", [(1, 1, 1), (37, 1000, 1), (300, 257, 3), (5, 16384, 5), (24, 64, 0)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_loop_kernels(N, H, B, dt):
    """The kernels for any width and alignment, which otherwise only very wide
    rows reach, on ordinary ones."""
    c = join_inputs(N, H, DT[dt], torch.float32, B, seed=N)
    table = rnd((20, H), 3, DT[dt])
    tokens = torch.arange(N, device=DEV) % 20
    _lib.set_kernel_path(2)
    try:
        out = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], 1e-5, residual_scale=0.75)
        grad, rpost, rpre = run_join_grad(c, True, True)
        y, h, r = nl.embedding_rms(tokens, table, c["gpre"], 1e-5, 1.5)
    finally:
        _lib.set_kernel_path(0)
    torch.cuda.synchronize()
    check_join(c, out, 1e-5, 0.75, True, True)
    check_join_grad(c, grad, rpost, rpre, 0.75)
    ry, rh, rr = S.lookup_forward(tokens.tolist(), n64(table), 1.5, n64(c["gpre"]), 1e-5)
    close(h, rh, U * np.abs(rh), "h")
    close(y, ry, 2 * steps(H) * U * np.abs(ry), "y")


def test_offsets_past_32_bits():
    """Rows, and rows of a table, more than 2^31 elements apart."""
    N, H, ld = 3, 1040, 1_200_000_000
    small = join_inputs(N, H, torch.bfloat16, torch.bfloat16, 1, seed=8)

    def far(t):
        buf = torch.empty((N - 1) * ld + H, dtype=t.dtype, device=DEV)
        view = buf.as_strided((N, H), (ld, 1))
        view.copy_(t)
        return view

    c = {k: far(v) if k in ("x", "res") else v for k, v in small.items()}
    want = nl.sandwich_rms(small["x"], small["res"], small["gpost"], small["gate"], small["gpre"])
    got = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], h_out=far(small["x"]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del got
    g, rpost, rpre = run_join_grad(small, True, True)
    f = nl.sandwich_rms_grad(small["dy"], c["x"], c["res"], rpost, rpre, c["gpost"], c["gate"], c["gpre"], small["dh"],
                             residual_scale=0.75)
    assert all(torch.equal(a, b) for a, b in zip(f, g))
    tokens = torch.tensor([2, 0, 2], device=DEV)
    assert torch.equal(nl.embedding_lookup(tokens, c["x"]), small["x"][tokens])
    out = far(small["x"])
    nl.embedding_grad(small["dy"], tokens, N, out=out)
    assert torch.equal(out.contiguous(), nl.embedding_grad(small["dy"], tokens, N))


def test_calls_at_once_on_two_streams():
    """Calls that overlap on the GPU do not meet: each has its own workspace."""
    c = [join_inputs(2000, 1024, torch.bfloat16, torch.bfloat16, 8, seed=i) for i in range(2)]
    tok = [torch.from_numpy(make_tokens("skewed", 2000, 500 + i)).to(DEV) for i in range(2)]
    st = [torch.cuda.Stream() for _ in range(2)]
    want = [(run_join_grad(c[i], True, True)[0], nl.embedding_grad(c[i]["dy"], tok[i], 500 + i)) for i in range(2)]
    rp = [[torch.from_numpy(S._rstd(n64(c[i][k]), 1e-5)).float().to(DEV) for k in ("x", "res")] for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                d = c[i]
                got[i].append((nl.sandwich_rms_grad(d["dy"], d["x"], d["res"], *rp[i], d["gpost"], d["gate"], d["gpre"],
                                                    d["dh"], residual_scale=0.75),
                               nl.embedding_grad(d["dy"], tok[i], 500 + i)))
    torch.cuda.synchronize()
    for i in range(2):
        for g, e in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i][0])) and torch.equal(e, want[i][1])


def test_expanded_and_permuted_tensors_are_refused():
    x = torch.zeros((6, 64), device=DEV, dtype=torch.bfloat16)
    with pytest.raises(nl.NormError):
        nl.sandwich_rms(x, x[:1].expand(6, 64))
    with pytest.raises(nl.NormError):
        nl.sandwich_rms(x, x.clone(), gate=x[:1].expand(3, 64))
    t = torch.zeros((4, 5, 64), device=DEV)
    with pytest.raises(ValueError, match="flatten"):
        nl.sandwich_rms(t.transpose(0, 1), torch.zeros((5, 4, 64), device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        nl.sandwich_rms(t[..., ::2], t[..., ::2])
    with pytest.raises(TypeError):
        nl.sandwich_rms(t.double(), t.double())


def test_device_words_of_the_far_kernels_stay_clear():
    assert _lib.device_errors() == 0


@pytest.mark.parametrize("N,H", [(1, 256), (8, 4096), (700, 1024), (4000, 512), (300, 8192)])
def test_calls_close_behind_one_another(N, H):
    """Kernels start while the ones before them drain: what those wrote (rows,
    parameters, the stream in place, the gradient's inputs) has to be seen, and
    what they read not overwritten.  The same run with a wait after every call
    gives the same bits."""
    dt = torch.bfloat16
    src = [rnd((N, H), i, dt) for i in range(3)]
    table = rnd((64, H), 7, dt)
    tokens = torch.from_numpy(make_tokens("skewed", N, 64)).to(DEV)

    def go(wait):
        def sync():
            if wait:
                torch.cuda.synchronize()
        x, stream, out = src[0].clone(), src[1].clone(), torch.empty_like(src[0])
        gamma, gate = torch.ones(H, device=DEV, dtype=dt), torch.full((H,), 0.5, device=DEV, dtype=dt)
        seen = []
        for i in range(40):
            x.copy_(src[i % 3])
            sync()
            gamma.mul_(1.0 + 0.01 * (i % 5))
            sync()
            y, h, rp, rq = nl.sandwich_rms(x, stream, gamma, gate, gamma, residual_scale=0.5, h_out=stream, out=out)
            sync()
            y2, h2, _, _ = nl.sandwich_rms(y, h, gamma, gate, gamma, residual_scale=0.5)
            sync()
            dx, dr, a, b, c = nl.sandwich_rms_grad(y2, x, h, rp, rq, gamma, gate, gamma, h2, residual_scale=0.5)
            sync()
            x.zero_()
            sync()
            e, eh, _ = nl.embedding_rms(tokens, table, gamma)
            sync()
            t = nl.embedding_grad(dr, tokens, 64)
            sync()
            table.copy_(t)
            sync()
            gamma.copy_(torch.ones_like(gamma))
            sync()
            seen += [y.clone(), h.clone(), y2, dx, dr, a, b, c, e, eh, t]
        torch.cuda.synchronize()
        return seen

    keep = table.clone()
    want = go(True)
    for _ in range(2):
        table.copy_(keep)
        assert all(torch.equal(a, b) for a, b in zip(want, go(False)))


def _expanded(B, T, H, dt):
    """(B, T, H) tensors over fewer rows: a row a sequence, the rows of one
    sequence, one row."""
    t = torch.zeros((B, T, H), device=DEV, dtype=dt)
    return [t[:, :1].expand(B, T, H), t[:1].expand(B, T, H), t[:1, :1].expand(B, T, H)]


def test_expanded_rows_of_more_dims_are_refused():
    """Every row tensor of every call, before anything is launched (the views
    themselves are checked on the CPU)."""
    B, T, H, V = 4, 6, 64, 10
    x = torch.zeros((B, T, H), device=DEV, dtype=torch.bfloat16)
    r = torch.ones(B * T, device=DEV)
    tok = torch.zeros((B, T), device=DEV, dtype=torch.int64)
    table = torch.zeros((V, H), device=DEV, dtype=torch.bfloat16)
    grad = dict(dy=x, x=x, h=x, rstd_post=r, rstd_pre=r, dh_in=x)
    for e in _expanded(B, T, H, torch.bfloat16):
        calls = [lambda: nl.sandwich_rms(e, x), lambda: nl.sandwich_rms(x, e), lambda: nl.sandwich_rms(x, x, gate=e),
                 lambda: nl.sandwich_rms(x, x, h_out=e), lambda: nl.sandwich_rms(x, x, out=e),
                 lambda: nl.embedding_lookup(tok, table, out=e), lambda: nl.embedding_rms(tok, table, h_out=e),
                 lambda: nl.embedding_rms(tok, table, out=e), lambda: nl.embedding_grad(e, tok, V)]
        calls += [lambda k=k: nl.sandwich_rms_grad(**{**grad, k: e}) for k in ("dy", "x", "h", "dh_in")]
        calls += [lambda k=k: nl.sandwich_rms_grad(**grad, **{k: e}) for k in ("gate", "dx", "dres")]
        for i, call in enumerate(calls):
            with pytest.raises((ValueError, nl.NormError)):
                call()
                raise AssertionError(i)


def test_the_gradient_of_a_sum_over_tokens():
    """y.sum(1) with a factor a sequence sends back a row a sequence, expanded
    over its tokens: refused as it is, taken after contiguous()."""
    B, T, H = 4, 6, 64
    c = join_inputs(B * T, H, torch.float32, torch.float32, 1)
    y = torch.zeros((B, T, H), device=DEV, requires_grad=True)
    dy, = torch.autograd.grad((y.sum(1) * rnd((B, H), 3, torch.float32)).sum(), y)
    assert dy.stride() == (H, 0, 1)
    rpost, rpre = (torch.from_numpy(S._rstd(n64(c[k]), 1e-5)).float().to(DEV) for k in ("x", "res"))

    def call(dy):
        return nl.sandwich_rms_grad(dy, c["x"], c["res"], rpost, rpre, c["gpost"], c["gate"], c["gpre"], c["dh"],
                                    residual_scale=0.75)
    with pytest.raises(ValueError, match="flatten"):
        call(dy)
    with pytest.raises(ValueError, match="flatten"):
        nl.embedding_grad(dy, torch.zeros((B, T), device=DEV, dtype=torch.int64), 3)
    c["dy"] = dy.contiguous().view(B * T, H)
    check_join_grad(c, call(dy.contiguous()), rpost, rpre, 0.75)


@pytest.mark.parametrize("gates", [0, 1])
@pytest.mark.parametrize("N,H,dt", [(24000, 96, "bf16"), (24000, 97, "f16"), (24000, 130, "f32"), (24001, 61, "f32"),
                                    (8000, 513, "f16"), (3000, 2057, "f16"), (2000, 4096, "bf16"), (1000, 5121, "f16"),
                                    (700, 4097, "f32"), (500, 16384, "bf16")])
def test_join_grad_refills_its_buffers(N, H, dt, gates):
    """Six rows and more a row group, which has at most four buffers: rows of
    one warp and of several, aligned and not (whose ends are loaded early and
    stored a row later), in one CTA and in clusters."""
    c = join_inputs(N, H, DT[dt], DT[dt], gates, seed=N + gates)
    out, rpost, rpre = run_join_grad(c, True, True)
    check_join_grad(c, out, rpost, rpre, 0.75)
    again, _, _ = run_join_grad(c, True, True)
    assert all(torch.equal(a, b) for a, b in zip(out, again) if a is not None)


def test_lookup_grad_one_workspace_for_smaller_batches():
    H, V = 72, 400
    ws = torch.empty(_lib.load().embedding_grad_workspace_bytes(10000, H), device=DEV, dtype=torch.uint8)
    dh = rnd((10000, H), 1, torch.bfloat16)
    for n in (10000, 8193, 8192, 8000, 4097, 4096, 33, 1):
        tok = torch.from_numpy(make_tokens("skewed", n, V)).to(DEV)
        out = nl.embedding_grad(dh[:n], tok, V, workspace=ws)
        assert torch.equal(out, nl.embedding_grad(dh[:n], tok, V))


@pytest.mark.parametrize("H", [64, 1001, 5120])
def test_join_tiny_eps(H):
    """A block output whose squares underflow but whose norm does not: with
    eps = 1e-30 values of 1e-23 become 1e-8, whose squares count against eps."""
    x = torch.full((3, H), 1e-23, device=DEV)
    x[1] *= torch.sign(rnd((H,), 1, torch.float32))
    c = dict(x=x, res=torch.zeros_like(x), gpost=rnd((H,), 2, torch.float32, 1.0, 0.1), gate=None,
             gpre=rnd((H,), 3, torch.float32, 1.0, 0.1))
    out = nl.sandwich_rms(x, c["res"], c["gpost"], None, c["gpre"], 1e-30)
    check_join(c, out, 1e-30, 1.0, True, True)


def test_join_gates_of_an_empty_batch():
    """No sequences: no gate rows either, and gradients of those shapes."""
    x = torch.empty((0, 5, 64), device=DEV, dtype=torch.bfloat16)
    r = torch.empty((0, 5), device=DEV)
    gate = torch.empty((0, 1, 64), device=DEV, dtype=torch.bfloat16)
    y, h, a, b = nl.sandwich_rms(x, x, None, gate)
    assert y.shape == h.shape == x.shape and a.numel() == b.numel() == 0
    dx, dr, dp, dg, dn = nl.sandwich_rms_grad(x, x, x, r, r, None, gate)
    assert dx.shape == dr.shape == x.shape and dg.shape == gate.shape
    assert dp.shape == dn.shape == (64,) and not dp.any() and not dn.any()
    some = torch.zeros((5, 64), device=DEV, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="divide"):
        nl.sandwich_rms(some, some, None, gate)


@pytest.mark.parametrize("N,H,dt", [(30000, 64, "bf16"), (30000, 65, "f16"), (30001, 24, "f32"), (4000, 1001, "f32"),
                                    (4000, 4096, "bf16"), (2500, 2057, "f16"), (1000, 16384, "bf16")])
def test_lookup_several_rows_a_group(N, H, dt):
    """Three rows and more a row group: the row and the token after the one at
    work are asked for ahead, bad tokens among them."""
    V = 300
    table = rnd((V, H), H, DT[dt])
    gamma = rnd((H,), 2, DT[dt], 1.0, 0.1)
    tokens = make_tokens("skewed", N, V)
    tokens[::97] = V
    tokens[5::1009] = -1
    tok = torch.from_numpy(tokens).to(DEV)
    y, h, rstd = nl.embedding_rms(tok, table, gamma, 1e-5, 1.5)
    only = nl.embedding_lookup(tok.int(), table, 1.5)
    torch.cuda.synchronize()
    assert torch.equal(only, h) and _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_TOKEN
    # a row depends on its token alone: the oracle's row of each token, and zeros
    ry, rh, rr = S.lookup_forward(list(range(V)) + [V], n64(table), 1.5, n64(gamma), 1e-5)
    row = np.where((tokens < 0) | (tokens >= V), V, tokens)
    k = steps(H) * U
    close(h, rh[row], U * np.abs(rh[row]), "h")
    close(rstd, rr[row], k * rr[row], "rstd")
    close(y, ry[row], 2 * k * np.abs(ry[row]), "y")


@pytest.mark.parametrize("kind", KINDS + ["bad"])
@pytest.mark.parametrize("N,H,V,dt,odt,ld,it,off", [
    (40, 1040, 20000, "bf16", "bf16", 1040, torch.int64, 0), (600, 1040, 3000, "bf16", "bf16", 1040, torch.int64, 0),
    (601, 1040, 3000, "f16", "f16", 1048, torch.int32, 1), (333, 1041, 2000, "bf16", "bf16", 1041, torch.int64, 1),
    (500, 520, 4000, "f16", "f32", 523, torch.int32, 3), (300, 5000, 200, "f32", "f32", 5000, torch.int64, 0),
    (4, 1024, 700, "bf16", "f32", 1024, torch.int32, 0)])
def test_lookup_grad_marked_clearing(kind, N, H, V, dt, odt, ld, it, off):
    """Few tokens, rows of 2 KB and more: the rows that no token names are
    cleared beside the sums, by marks made from the tokens. The table's rows are
    aligned, padded or shifted, the tokens 16-byte aligned or not."""
    tokens = make_tokens("uniform" if kind == "bad" else kind, N, V)
    if kind == "bad":
        tokens[::3] = V
        tokens[1::7] = -5
    pad = V - 1 if kind == "padded" else -1
    buf = torch.zeros(N + off, device=DEV, dtype=it)
    tok = buf[off:]
    tok.copy_(torch.from_numpy(tokens))
    dh = rnd((N, H), N, DT[dt])
    view, whole, rest = padded(torch.full((V, H), 3.0, dtype=DT[odt], device=DEV), ld)
    out = nl.embedding_grad(dh, tok, V, 1.5, padding_idx=None if pad < 0 else pad, out=view)
    torch.cuda.synchronize()
    assert torch.all(whole[rest] == -77.0)
    assert _lib.device_errors() == (_lib.NORM_DEVICE_ERR_BAD_TOKEN if kind == "bad" else 0)
    d = n64(dh)
    ref = S.lookup_backward(d, tokens, V, 1.5, pad)
    terms = S.lookup_backward(np.abs(d), tokens, V, 1.5, pad)
    counts = np.bincount(tokens[(tokens >= 0) & (tokens < V)], minlength=V)
    close(out, ref, (40 + counts[:, None] / 8) * U * terms, "dtable")  # tiles of eight
    assert not out[torch.from_numpy((counts == 0) | (np.arange(V) == pad)).to(DEV)].any()


def test_lookup_grad_marks_in_several_ranges():
    """More table rows a clearing CTA than it marks at a time (8192)."""
    V, H = 5_300_000, 1024
    tokens = torch.tensor([0, 1, 8191, 8192, 8716, 8717, 8718, 3_000_000, V - 1, V - 1, 8192], device=DEV)
    dh = rnd((len(tokens), H), 1, torch.bfloat16)
    out = torch.full((V, H), 3.0, device=DEV, dtype=torch.bfloat16)
    nl.embedding_grad(dh, tokens, V, out=out)
    ids = tokens.unique()
    want = S.lookup_backward(n64(dh), torch.searchsorted(ids, tokens).tolist(), len(ids))
    close(out[ids], want, 4 * U * 2 * np.abs(want).max(), "dtable")
    out[ids] = 0
    assert not any(part.any() for part in out.split(500_000))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,H,B", [(300, 1024, 0), (301, 1001, 1), (96, 5120, 8), (40, 40008, 2)])
def test_join_without_parameters_and_stream_gradient(N, H, B, dt):
    """dh_in and the gammas left out: zeros and ones, with gradients of the ones."""
    c = join_inputs(N, H, DT[dt], DT[dt], B, seed=H)
    ones, c["dh"] = torch.ones(H, device=DEV), torch.zeros_like(c["x"])
    c["gpost"] = c["gpre"] = ones
    out = nl.sandwich_rms(c["x"], c["res"], None, c["gate"], None, 1e-5, residual_scale=0.75)
    check_join(c, out, 1e-5, 0.75, True, True)
    rpost, rpre = (torch.from_numpy(S._rstd(n64(c[k]), 1e-5)).float().to(DEV) for k in ("x", "res"))
    for p in (True, False):  # (without the norm after the block too)
        grad = nl.sandwich_rms_grad(c["dy"], c["x"], c["res"], rpost if p else None, rpre, None, c["gate"], None, None,
                                    residual_scale=0.75, param_dtype=torch.float32)
        check_join_grad(c, grad, rpost if p else None, rpre, 0.75)
        assert grad[4].dtype == torch.float32


@pytest.mark.parametrize("wdt,gdt", [("x", "f32"), ("f32", "x"), ("f32", "f32")])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,H,B", [(300, 1024, 1), (300, 1024, 4), (303, 1001, 3), (60, 16384, 5)])
def test_join_parameter_dtypes(N, H, B, dt, wdt, gdt):
    """Gammas in the rows' dtype with an fp32 gate, and the other way round."""
    wt, gt = (DT[dt if d == "x" else d] for d in (wdt, gdt))
    c = join_inputs(N, H, DT[dt], wt, B, seed=N, gdt=gt)
    out = nl.sandwich_rms(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], 1e-5, residual_scale=0.75)
    check_join(c, out, 1e-5, 0.75, True, True)
    out, rpost, rpre = run_join_grad(c, True, True)
    assert out[2].dtype == out[4].dtype == wt and out[3].dtype == gt
    check_join_grad(c, out, rpost, rpre, 0.75)


@pytest.mark.parametrize("H,dt", [(30208, "f16"), (30209, "f16"), (30272, "bf16"), (30280, "bf16"), (30720, "bf16"),
                                  (32768, "f16"), (32769, "f16"), (32768, "f32")])
def test_join_grad_widest_rows_with_gates_of_runs(H, dt):
    """Where several gate rows leave no room for two row buffers, the loop runs
    (half precision: past 30272 columns, 30208 in element accesses)."""
    c = join_inputs(12, H, DT[dt], torch.float32, 4, seed=H)
    out, rpost, rpre = run_join_grad(c, True, True)
    check_join_grad(c, out, rpost, rpre, 0.75)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_an_event_of_another_stream(captured):
    """What a call waits for besides the kernel before it in its own stream: an
    event behind long work elsewhere, copies and memsets. Eager, and as the edges
    of a graph."""
    N, H, V = 64, 1024, 50
    a = rnd((4096, 4096), 1, torch.bfloat16, std=0.02)
    src = rnd((N, H), 2, torch.bfloat16)
    table = rnd((V, H), 3, torch.bfloat16)
    tokens = torch.from_numpy(make_tokens("skewed", N, V)).to(DEV)
    x, res, tok, dy = torch.empty_like(src), torch.empty_like(src), torch.empty_like(tokens), torch.empty_like(src)
    stats = torch.ones(N, device=DEV)
    side = torch.cuda.Stream()

    def go():
        main = torch.cuda.current_stream()
        x.zero_()
        dy.zero_()
        tok.zero_()
        outs = []
        for i in range(3):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                b = a @ a
                for _ in range(3):
                    b = b @ a
                x.copy_(src * (i + 1) + 0 * b[:N, :H])
                dy.copy_(src + 0 * b[:N, :H])
                tok.copy_(tokens)
            res.copy_(src)   # the kernel before the call in its own stream ends long before the event
            main.wait_stream(side)
            y, h, _, _ = nl.sandwich_rms(x, res)
            side.wait_stream(main)
            with torch.cuda.stream(side):
                x.add_(b[:N, :H] * 0)
            main.wait_stream(side)
            outs += [y, h, *nl.sandwich_rms_grad(dy, x, h, stats, stats)]
            e, eh, _ = nl.embedding_rms(tok, table)
            tok.fill_(1)
            outs += [e, eh, nl.embedding_grad(dy, tok, V)]
            x.zero_()
            dy.zero_()
            tok.zero_()
        return outs

    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = go()
        for _ in range(3):
            g.replay()
    else:
        got = go()
    torch.cuda.synchronize()
    want = []
    for i in range(3):
        xs = src * (i + 1)
        y, h, _, _ = nl.sandwich_rms(xs, src)
        torch.cuda.synchronize()
        want += [y, h, *nl.sandwich_rms_grad(src, xs, h, stats, stats)]
        torch.cuda.synchronize()
        e, eh, _ = nl.embedding_rms(tokens, table)
        torch.cuda.synchronize()
        want += [e, eh, nl.embedding_grad(src, torch.ones_like(tokens), V)]
    for p, q in zip(got, want):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("x,gate", [((4, 6, 64), (1, 6, 64)), ((2, 3, 6, 64), (1, 3, 1, 64)),
                                    ((2, 3, 6, 64), (2, 1, 6, 64)), ((2, 3, 6, 64), (1, 3, 6, 64))])
def test_gates_of_positions_are_refused(x, gate):
    """Shapes that would broadcast over an outer dim are no runs of rows."""
    t, g = (torch.zeros(s, device=DEV) for s in (x, gate))
    r = torch.ones(t.numel() // 64, device=DEV)
    with pytest.raises(ValueError, match="run of consecutive rows"):
        nl.sandwich_rms(t, t, gate=g)
    with pytest.raises(ValueError, match="run of consecutive rows"):
        nl.sandwich_rms_grad(t, t, t, r, r, None, g)


@pytest.mark.parametrize("x,gate", [((4, 6, 64), (4, 1, 64)), ((4, 6, 64), (4, 6, 64)), ((4, 6, 64), (1, 1, 64)),
                                    ((1, 6, 64), (1, 6, 64)), ((2, 3, 6, 64), (2, 3, 1, 64)), ((4, 6, 64), (8, 1, 64)),
                                    ((4, 1, 6, 64), (4, 1, 1, 64)), ((4, 6, 64), (64,)), ((4, 6, 64), (1, 64))])
def test_gate_shapes_are_runs_of_rows(x, gate):
    t, res, g = rnd(x, 1, torch.float32), rnd(x, 2, torch.float32), rnd(gate, 3, torch.float32)
    N = t.numel() // 64
    rows = g.reshape(-1, 64).repeat_interleave(N // (g.numel() // 64), 0).reshape(x)
    y, h, _, _ = nl.sandwich_rms(t, res, gate=g, post_norm=False)
    want = res.double() + rows.double() * t.double()
    assert (h.double() - want).abs().max() <= 2 * U * (res.abs() + (rows * t).abs()).max()  # (the product and the sum)

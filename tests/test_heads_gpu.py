"""The per-head norm with the rotation by position on the GPU against the fp64
oracle.

Tolerances, from the arithmetic (U = 2^-24, half an fp32 step):

* sum(x^2) of a head: 8 serial additions of pairs in a lane, one between the
  pair's members and 5 tree levels, two roundings a term: 16 U relative.  rstd
  halves that and adds the mean's and eps' roundings and rsqrtf's two steps:
  13 U.  n = x rstd gamma: 15 U.  A rotated column is a sum of two products:
  3 U more.  KF = 20 steps of U on the magnitudes of its two terms.
* dx = rstd (w - x rstd^2 mean(w x)): w has 4 U on the magnitudes of u's terms,
  the sum 16 U more, rstd^2 26 U, products 4 U, rstd again 13 U: KB = 64.
* dgamma, a sum over rows: u x rstd has 18 U a term.  Units, one head of as many
  tokens as a warp has lane groups, are shared out evenly over the warps (2432 of
  them, or one unit each): a lane adds at most rows/256 + 4.  Then the CTA adds up
  8 warps of at most 32 groups, 256 in a row, and the partial rows 19 + 16 and 4
  levels: 300 in all.
* a value stored in fewer bits: half a step, on top.
"""

import numpy as np
import pytest
import torch

import rmsnorm_ln_fwd_gb300 as nl
from oracle import head_oracle as O
from rmsnorm_ln_fwd_gb300 import _lib, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
KF, KB = 20, 64
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


def rnd(shape, seed, dt, mean=0.0, std=1.0):
    return synth.normal(shape, seed, "x", mean=mean, std=std, dtype=dt).to(DEV)


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


def tables(rows, R, cdt=torch.float32):
    a = np.arange(rows)[:, None] * 1000.0 ** (-np.arange(R // 2) / max(1, R // 2))
    return torch.tensor(np.cos(a)).to(cdt).to(DEV), torch.tensor(np.sin(a)).to(cdt).to(DEV)


def make(B, T, hq, hk, D, R, dt, wdt=None, layout="separate", rows=None, positions="none", seed=0, cdt=torch.float32):
    """A dict of head_rms_rotary's arguments, and dyq, dyk."""
    dt = DT[dt]
    wdt = dt if wdt is None else DT[wdt]
    rows = rows or max(T, 64)

    def heads(H, s):
        if layout == "bhtd":
            return rnd((B, H, T, D), s, dt, std=1.5).transpose(1, 2)
        return rnd((B, T, H, D), s, dt, std=1.5)

    if layout == "fused":
        whole = rnd((B, T, (hq + 2 * hk) * D), seed, dt, std=1.5)
        q = whole[..., :hq * D].unflatten(-1, (hq, D))
        k = whole[..., hq * D:(hq + hk) * D].unflatten(-1, (hk, D)) if hk else None
    else:
        q, k = heads(hq, seed), heads(hk, seed + 1) if hk else None
    c = dict(q=q, k=k, gq=rnd((D,), seed + 2, wdt, 1.0, 0.2), gk=rnd((D,), seed + 3, wdt, 1.0, 0.2) if hk else None,
             cos=None, sin=None, pos=None, dyq=heads(hq, seed + 4), dyk=heads(hk, seed + 5) if hk else None)
    if R:
        c["cos"], c["sin"] = tables(rows, R, cdt)
        r = np.random.default_rng(seed)
        if positions == "shared":
            c["pos"] = torch.tensor(r.integers(0, rows, T), device=DEV)
        elif positions == "each":
            c["pos"] = torch.tensor(r.integers(0, rows, (B, T)), device=DEV, dtype=torch.int32)
    return c


def call(c, eps=1e-5, interleaved=False, **kw):
    return nl.head_rms_rotary(c["q"], c["k"], c["gq"], c["gk"], c["cos"], c["sin"], c["pos"], eps,
                              interleaved=interleaved, **kw)


def call_grad(c, eps=1e-5, interleaved=False, **kw):
    return nl.head_rms_rotary_grad(c["dyq"], c["dyk"], c["q"], c["k"], c["gq"], c["gk"], c["cos"], c["sin"], c["pos"],
                                   eps, interleaved=interleaved, **kw)


def token_tables(c, x):
    """cos and sin of each token, and which tokens have them."""
    B, T = x.shape[0], x.shape[1]
    if c["cos"] is None:
        return None, None, np.ones(B * T, bool)
    p = np.broadcast_to(np.arange(T) if c["pos"] is None else c["pos"].cpu().numpy(), (B, T)).reshape(-1)
    good = (p >= 0) & (p < c["cos"].shape[0])
    at = np.where(good, p, 0)
    return n64(c["cos"])[at], n64(c["sin"])[at], good


def flat(x):
    return n64(x).reshape(-1, *x.shape[-2:])


def check(c, out, eps, interleaved, what=""):
    for side, y in (("q", out[0]), ("k", out[1])):
        x = c[side]
        if x is None:
            assert y is None
            continue
        assert y.shape == x.shape and y.dtype == x.dtype
        cos, sin, good = token_tables(c, x)
        g = n64(c["g" + side])
        ref = O.head_forward(flat(x), g, cos, sin, eps, interleaved, good)
        n = np.abs(flat(x) * O.head_rstd(flat(x), eps) * (1.0 if g is None else g))
        # magnitudes of the terms: |a||cos| + |b||sin| for both members
        terms = n if cos is None else O.turn(n, np.abs(cos), -np.abs(sin), interleaved)
        if cos is not None:
            terms = np.maximum(terms, O.turn(n, np.abs(cos), np.abs(sin), interleaved))
        close(y, ref.reshape(y.shape), (KF * U * np.abs(terms)).reshape(y.shape), f"{what}{side}")


def check_grad(c, out, eps, interleaved, what=""):
    for side, dx, dg in (("q", out[0], out[2]), ("k", out[1], out[3])):
        x = c[side]
        if x is None:
            assert dx is None and dg is None
            continue
        cos, sin, good = token_tables(c, x)
        g, X, dy = n64(c["g" + side]), flat(x), flat(c["dy" + side])
        rdx, rdg = O.head_backward(dy, X, g, cos, sin, eps, interleaved, good)
        gg = np.ones(X.shape[-1]) if g is None else np.abs(g)
        su = np.abs(dy)
        if cos is not None:
            su = np.maximum(O.turn(su, np.abs(cos), -np.abs(sin), interleaved), O.turn(su, np.abs(cos), np.abs(sin), interleaved))
        su = np.abs(su) * good[:, None, None]
        r = O.head_rstd(X, eps)
        terms = r * (su * gg + np.abs(X) * r * r * (su * gg * np.abs(X)).mean(-1, keepdims=True))
        close(dx, rdx.reshape(dx.shape), (KB * U * terms).reshape(dx.shape), f"{what}d{side}")
        if dg is not None:
            rows = X.shape[0] * X.shape[1]
            K = 18 + 304 + rows / 256
            close(dg, rdg, K * U * (su * np.abs(X) * r).sum((0, 1)), f"{what}dgamma_{side}")


# B, T, hq, hk, D, R
SHAPES = [(1, 1, 1, 1, 1, 0), (1, 1, 1, 0, 2, 2), (1, 1, 32, 8, 128, 128), (2, 3, 4, 2, 64, 64), (3, 5, 6, 3, 80, 32),
          (1, 7, 9, 3, 96, 48), (2, 2, 5, 1, 80, 40), (1, 9, 2, 2, 256, 256), (1, 3, 2, 1, 512, 512), (1, 4, 3, 3, 33, 10),
          (2, 3, 2, 2, 7, 6), (1, 2, 2, 1, 500, 250), (1, 301, 4, 4, 112, 56), (5, 67, 8, 2, 128, 64), (1, 40, 7, 2, 16, 16),
          (2, 16, 3, 1, 48, 0), (1, 2, 70, 9, 24, 24)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradient(shape, dt, interleaved):
    B, T, hq, hk, D, R = shape
    layout = ("separate", "fused", "bhtd")[(T + D) % 3]
    positions = ("none", "shared", "each")[(B + hq + T) % 3]
    c = make(*shape, dt, wdt="f32" if D % 3 else None, layout=layout, positions=positions, seed=D + T)
    out = call(c, interleaved=interleaved)
    grad = call_grad(c, interleaved=interleaved)
    torch.cuda.synchronize()
    check(c, out, 1e-5, interleaved)
    check_grad(c, grad, 1e-5, interleaved)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("layout", ["separate", "fused", "bhtd"])
def test_layouts(dt, layout):
    c = make(2, 37, 8, 4, 64, 64, dt, layout=layout, positions="each", seed=3)
    check(c, call(c), 1e-5, False)
    check_grad(c, call_grad(c), 1e-5, False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["separate", "fused", "bhtd"])
def test_in_place_has_the_same_bits(dt, layout):
    c = make(2, 19, 6, 2, 96, 48, dt, layout=layout, seed=4)
    fresh, grads = call(c), call_grad(c)
    dyq, dyk = c["dyq"].clone(memory_format=torch.preserve_format), c["dyk"].clone(memory_format=torch.preserve_format)
    got = call_grad({**c, "dyq": dyq, "dyk": dyk}, dq=dyq, dk=dyk)
    assert got[0] is dyq or got[0].data_ptr() == dyq.data_ptr()
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    whole = c["q"]._base.clone() if layout == "fused" else None
    q, k = c["q"], c["k"]
    call(c, q_out=q, k_out=k)
    assert torch.equal(q, fresh[0]) and torch.equal(k, fresh[1])
    if layout == "fused":  # the values behind the keys stay as they were
        assert torch.equal(q._base[..., -2 * 96:], whole[..., -2 * 96:])


@pytest.mark.parametrize("order", ["decode", "tokens first", "heads first", "one sequence"])
def test_in_place_on_a_fused_projection(order):
    """Queries and keys whose elements are between one another's, in the layouts in which projections leave them."""
    hq, hk, D = 6, 2, 64
    B, T = {"decode": (8, 1), "one sequence": (1, 21)}.get(order, (3, 11))
    if order == "tokens first":    # (T, B, heads * D)
        base = rnd((T, B, hq + 2 * hk, D), 40, torch.bfloat16).transpose(0, 1)
    elif order == "heads first":   # (B, heads, T, D)
        base = rnd((B, hq + 2 * hk, T, D), 40, torch.bfloat16).transpose(1, 2)
    else:
        base = rnd((B, T, hq + 2 * hk, D), 40, torch.bfloat16)
    q, k, v = base[:, :, :hq], base[:, :, hq:hq + hk], base[:, :, hq + hk:].clone()
    c = dict(q=q, k=k, gq=rnd((D,), 41, torch.bfloat16, 1.0, 0.2), gk=rnd((D,), 42, torch.bfloat16, 1.0, 0.2), pos=None)
    c["cos"], c["sin"] = tables(64, D)
    want = call(c)
    call(c, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(base[:, :, hq + hk:], v)
    # into another's place: the keys' heads over the last query heads
    with pytest.raises(nl.NormError):
        call(c, q_out=q, k_out=base[:, :, hq - 1:hq - 1 + hk])


@pytest.mark.parametrize("D,R,dt", [(64, 64, "bf16"), (80, 20, "f16"), (48, 0, "f32")])
def test_in_place_where_a_heads_query_key_and_value_are_side_by_side(D, R, dt):
    """(B, T, heads, 3, D), forward in place, and the gradients as parts of such a tensor."""
    B, T, H = 2, 13, 5
    base, grads = (rnd((B, T, H, 3, D), s, DT[dt]) for s in (50, 51))
    q, k, v = (base[:, :, :, i] for i in range(3))
    c = dict(q=q, k=k, gq=rnd((D,), 52, DT[dt], 1.0, 0.2), gk=rnd((D,), 53, DT[dt], 1.0, 0.2), cos=None, sin=None, pos=None,
             dyq=grads[:, :, :, 0], dyk=grads[:, :, :, 1])
    if R:
        c["cos"], c["sin"] = tables(64, R)
    want, dwant, v, dv = call(c), call_grad(c), v.clone(), grads[:, :, :, 2].clone()
    check(c, want, 1e-5, False)
    into = torch.full_like(base, 3.0)
    got = call_grad(c, dq=into[:, :, :, 0], dk=into[:, :, :, 1])
    for a, b in zip(got, dwant):
        assert torch.equal(a, b)
    assert bool((into[:, :, :, 2] == 3.0).all())
    call_grad(c, dq=c["dyq"], dk=c["dyk"])
    assert torch.equal(c["dyq"], dwant[0]) and torch.equal(c["dyk"], dwant[1]) and torch.equal(grads[:, :, :, 2], dv)
    call(c, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(base[:, :, :, 2], v)
    with pytest.raises(nl.NormError):  # a query's last column
        call(c, q_out=q, k_out=base.view(B, T, H, 3 * D)[..., D - 1:2 * D - 1])


def test_outputs_in_other_layouts_and_margins():
    c = make(2, 11, 4, 2, 64, 32, "bf16", layout="fused", seed=5)
    want = call(c)
    # (B, H, T, D) tensors inside larger ones, whose rest must stay
    base = torch.full((2, 6, 13, 72), 7.0, device=DEV, dtype=torch.bfloat16)
    qo, ko = base[:, :4, 1:12, 4:68].transpose(1, 2), base[:, 4:, 1:12, 4:68].transpose(1, 2)
    call(c, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    keep = torch.ones_like(base, dtype=torch.bool)
    keep[:, :, 1:12, 4:68] = False
    assert bool((base[keep] == 7.0).all())
    # the same for the gradient, from expanded gradients
    one = rnd((64,), 9, torch.bfloat16)
    c["dyq"], c["dyk"] = one.expand(2, 11, 4, 64), one.expand(2, 11, 2, 64)
    base.fill_(7.0)
    got = call_grad(c, dq=qo, dk=ko)
    check_grad(c, got, 1e-5, False)
    assert bool((base[keep] == 7.0).all())


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shifted_addresses(dt, off):
    c = make(1, 21, 4, 2, 64, 64, dt, seed=6)

    def shift(t):
        flat = torch.empty(t.numel() + 16, device=DEV, dtype=t.dtype)
        v = flat[off:off + t.numel()].view(t.shape)
        return v.copy_(t)

    want, grads = call(c), call_grad(c)
    d = {**c, **{n: shift(c[n]) for n in ("q", "k", "dyq", "dyk", "gq", "gk")}}
    for a, b in zip(call(d) + call_grad(d)[:2], want + grads[:2]):
        assert torch.equal(a, b)
    cs = torch.empty(64, 65, device=DEV)  # table rows that no 16-byte access fits
    cos, sin = cs[:, 1:33].copy_(c["cos"]), cs[:, 33:].copy_(c["sin"])
    assert torch.equal(call({**c, "cos": cos, "sin": sin})[0], want[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_tables_in_the_rows_dtype_and_fused(interleaved):
    c = make(2, 23, 4, 2, 80, 40, "bf16", positions="each", cdt=torch.bfloat16, seed=7)
    check(c, call(c, interleaved=interleaved), 1e-5, interleaved)
    check_grad(c, call_grad(c, interleaved=interleaved), 1e-5, interleaved)
    c = make(2, 23, 4, 2, 80, 40, "bf16", positions="each", seed=7)
    want = call(c, interleaved=interleaved)
    cache = torch.cat([c["cos"], c["sin"]], 1)
    got = call({**c, "cos": cache[:, :20], "sin": cache[:, 20:]}, interleaved=interleaved)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_gamma_no_keys_no_rotation():
    c = make(2, 9, 3, 2, 64, 64, "f32", seed=8)
    c["gq"] = None
    check(c, call(c), 1e-5, False)
    g = call_grad(c)
    check_grad(c, g, 1e-5, False)
    assert g[2].dtype == torch.float32
    d = {**c, "gk": None}
    g = call_grad({**d, **{n: c[n].bfloat16() for n in ("q", "k", "dyq", "dyk")}}, param_dtype=torch.float32)
    assert g[2].dtype == g[3].dtype == torch.float32 and g[0].dtype == torch.bfloat16
    alone = {**c, "k": None, "dyk": None, "gk": None}
    assert torch.equal(call(alone)[0], call(c)[0]) and call(alone)[1] is None
    assert call_grad(alone)[3] is None
    plain = {**c, "cos": None, "sin": None}
    check(plain, call(plain), 1e-5, False)
    check_grad(plain, call_grad(plain), 1e-5, False)
    only = call_grad(c, need_param_grads=False)
    full = call_grad(c)
    assert only[2] is None and torch.equal(only[0], full[0]) and torch.equal(only[1], full[1])


def test_three_dims_are_one_sequence():
    c = make(1, 31, 4, 2, 64, 64, "bf16", positions="each", seed=9)
    want, grads = call(c), call_grad(c)
    d = {n: None if t is None else (t if t.dim() < 3 else t[0]) for n, t in c.items()}
    d["pos"] = c["pos"][0]
    for a, b in zip(call(d) + call_grad(d), want + grads):
        assert torch.equal(a.reshape(b.shape), b)
    # int64, strided and shared positions
    wide = torch.zeros(31, 3, device=DEV, dtype=torch.long)
    wide[:, 1] = c["pos"][0]
    assert torch.equal(call({**d, "pos": wide[:, 1]})[0], want[0][0])
    two = {n: None if t is None else (torch.cat([t, t]) if t.dim() == 4 else t) for n, t in c.items()}
    for pos in (c["pos"][0], c["pos"], c["pos"].expand(2, 31)):
        assert torch.equal(call({**two, "pos": pos})[0][1], want[0][0])


def test_empty_calls():
    for B, T in ((0, 4), (2, 0)):
        c = make(1, 4, 3, 2, 32, 32, "bf16")
        d = {n: None if t is None else (t if t.dim() < 4 else t[:, :T] if T == 0 else t[:B]) for n, t in c.items()}
        out = call(d)
        assert out[0].numel() == out[1].numel() == 0
        g = call_grad(d)
        assert g[0].numel() == 0 and not g[2].any() and not g[3].any()


def test_positions_outside_the_table():
    for idt in (torch.int32, torch.int64):
        c = make(2, 5, 4, 2, 64, 64, "f32", rows=50, positions="each", seed=10)
        c["pos"] = c["pos"].to(idt)
        c["pos"][0, 1], c["pos"][1, 3], c["pos"][1, 4] = -1, 50, torch.iinfo(idt).min
        _lib.device_errors()
        out = call(c)
        torch.cuda.synchronize()
        assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_POSITION
        check(c, out, 1e-5, False)
        assert not out[0][0, 1].any() and not out[1][1, 3].any()
        g = call_grad(c)
        torch.cuda.synchronize()
        assert _lib.device_errors() == _lib.NORM_DEVICE_ERR_BAD_POSITION
        check_grad(c, g, 1e-5, False)
        assert not g[0][1, 4].any()


def test_zero_and_far_heads():
    c = make(1, 6, 4, 2, 64, 64, "f32", seed=11)
    c["q"][0, 0] = 0.0                      # rstd = 1 / sqrt(eps)
    c["q"][0, 1] *= 1e-18                   # squares underflow
    c["q"][0, 2] *= 1e15
    c["k"][0, 3, 1] = 0.0
    check(c, call(c), 1e-5, False)
    out = call({**c, "dyq": c["dyq"]})
    assert not out[0][0, 0].any()
    check_grad(c, call_grad(c), 1e-5, False)


def test_a_head_that_is_not_finite_stays_alone():
    c = make(1, 6, 4, 2, 64, 32, "bf16", seed=12)
    want = call(c)
    c["q"][0, 2, 1, 5] = float("nan")
    c["q"][0, 3, 0, 40] = float("inf")
    got = call(c)
    bad = torch.zeros_like(got[0], dtype=torch.bool)
    bad[0, 2, 1] = bad[0, 3, 0] = True
    assert torch.equal(got[0][~bad], want[0][~bad]) and torch.equal(got[1], want[1])
    assert bool(got[0][0, 2, 1].isnan().all())
    # an infinite column: the norm is infinite, the others 0, whatever their pair (column 40 is not rotated)
    assert bool(got[0][0, 3, 0, 40].isnan()) and int(got[0][0, 3, 0].isnan().sum()) == 1


@pytest.mark.parametrize("shape,dt", [((4, 517, 32, 4, 128, 128), "bf16"), ((1, 2000, 16, 16, 64, 32), "f16"),
                                      ((1, 700, 8, 2, 256, 256), "f32"), ((1, 3000, 1, 1, 80, 80), "bf16")])
def test_many_tokens(shape, dt):
    """Warps that take several tokens, and every CTA of the gradient."""
    c = make(*shape, dt, wdt="f32", layout="fused", positions="each", seed=13)
    check(c, call(c), 1e-5, False)
    g = call_grad(c)
    check_grad(c, g, 1e-5, False)
    again = call_grad(c)
    for a, b in zip(g, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["plain", "interleaved", "unaligned table", "table of the rows' type"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 9001, 1, 0, 64, 64), (1, 9001, 1, 1, 16, 16), (3, 1501, 2, 0, 128, 64), (1, 5003, 5, 1, 128, 128),
                                   (1, 1999, 8, 2, 192, 192), (2, 997, 3, 1, 192, 96), (1, 1201, 1, 0, 500, 250), (7, 643, 2, 1, 48, 0)])
def test_few_heads_and_many_tokens(shape, dt, kind):
    """Warps that take blocks of tokens, or parts of them, one after another, while the angles of the next ones arrive."""
    R = shape[-1]
    own = kind == "table of the rows' type" and dt != "f32"
    c = make(*shape, dt, wdt="f32", layout="fused", positions="each", seed=sum(shape),
             cdt=DT[dt] if own else torch.float32)
    if R and kind == "unaligned table":
        rows = c["cos"].shape[0]
        both = torch.empty(rows, R + 1, device=DEV)
        c["cos"], c["sin"] = both[:, 1:R // 2 + 1].copy_(c["cos"]), both[:, R // 2 + 1:].copy_(c["sin"])
    if R:
        c["pos"][-1, -2], c["pos"][0, 5] = -3, c["cos"].shape[0]
    _lib.device_errors()
    pairs = kind == "interleaved"
    check(c, call(c, interleaved=pairs), 1e-5, pairs)
    check_grad(c, call_grad(c, interleaved=pairs), 1e-5, pairs)
    assert _lib.device_errors() == (_lib.NORM_DEVICE_ERR_BAD_POSITION if R else 0)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("D,R", [(80, 20), (84, 84), (64, 12), (20, 20), (36, 4), (16, 4), (80, 32), (100, 100), (256, 252), (160, 160),
                                 (144, 144), (40, 40), (72, 8), (60, 20), (68, 10), (24, 0), (88, 48), (476, 476), (44, 36)])
def test_columns_of_every_access_and_lanes_of_every_number(D, R, dt):
    """Halves that start at any multiple, lanes a head that are no power of two, at addresses of 16 and of 8 bytes."""
    c = make(3, 59, 3, 2, D, R, dt, wdt="f32", positions="each", seed=D + R)
    if R:
        c["pos"][1, 17] = -1
    want, grads = call(c), call_grad(c)
    check(c, want, 1e-5, False)
    check_grad(c, grads, 1e-5, False)
    for off in (8 // c["q"].element_size(), 1):

        def shift(t):
            flat = torch.full((t.numel() + 32,), 3.0, device=DEV, dtype=t.dtype)
            v = flat[off:off + t.numel()].view(t.shape)
            return v.copy_(t)

        d = {**c, **{n: shift(c[n]) for n in ("q", "k", "dyq", "dyk")}}
        q, k = torch.full_like(shift(c["q"]), 5.0), shift(torch.full_like(c["k"], 5.0))
        got = call(d, q_out=q, k_out=k)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        base = k._base
        assert bool((base[:off] == 3.0).all()) and bool((base[off + k.numel():] == 3.0).all())
        for a, b in zip(call_grad(d, dk=k), grads):
            assert torch.equal(a, b)
        assert bool((base[:off] == 3.0).all()) and bool((base[off + k.numel():] == 3.0).all())
    _lib.device_errors()


def test_an_infinite_column_beside_narrow_halves():
    """A column that is not rotated, in the same lane or the next one, and whatever a table's other columns hold."""
    for D, R in ((80, 20), (80, 40), (64, 32)):
        c = make(1, 6, 4, 2, D, R, "bf16", seed=D)
        want = call(c)
        c["q"][0, 3, 0, R + 1] = float("inf")
        got = call(c)
        assert torch.equal(got[0][0, 3, 1:], want[0][0, 3, 1:]) and torch.equal(got[1], want[1])
        assert bool(got[0][0, 3, 0, R + 1].isnan()) and int(got[0][0, 3, 0].isnan().sum()) == 1
        wide = torch.full((2, c["cos"].shape[0], R), float("nan"), device=DEV)
        wide[:, :, :R // 2] = torch.stack([c["cos"], c["sin"]])
        got = call({**c, "cos": wide[0, :, :R // 2], "sin": wide[1, :, :R // 2]})
        assert torch.equal(got[0][0, 4], want[0][0, 4]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    """Heads past 2^31 elements: repeated tokens have the bits of the first."""
    free = torch.cuda.mem_get_info()[0]
    if free < 30 << 30:
        pytest.skip("needs 30 GB")
    T, H, D = 140_000, 128, 128
    assert T * H * D > 2 ** 31
    one = rnd((1, H, D), 1, torch.bfloat16)
    q = one.expand(T, H, D).contiguous()
    g = rnd((D,), 2, torch.bfloat16, 1.0, 0.1)
    cos, sin = tables(4, D)
    pos = torch.full((T,), 3, device=DEV)
    y, _ = nl.head_rms_rotary(q, None, g, None, cos, sin, pos)
    assert bool((y == y[:1]).all())
    dx, _, dg, _ = nl.head_rms_rotary_grad(q, None, q, None, g, None, cos, sin, pos, param_dtype=torch.float32, dq=y)
    assert bool((dx == dx[:1]).all())
    _, _, d1, _ = nl.head_rms_rotary_grad(one, None, one, None, g.float().bfloat16(), None, cos, sin, pos[:1])
    # T times the first token's: each sum's rounding to bf16, half a step, and fp32 steps
    assert torch.allclose(dg.float(), T * d1.float(), rtol=2 * 2.0 ** -8, atol=T * 2.0 ** -8 * float(d1.float().abs().mean()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk,D,R,off", [(3, 2, 128, 128, 0), (3, 1, 80, 40, 0), (2, 2, 80, 20, 4), (2, 1, 33, 10, 0), (1, 0, 64, 64, 1)])
def test_sequences_more_than_32_bits_apart(hq, hk, D, R, off, interleaved):
    """Two sequences 2^31 elements apart, queries and keys, in every width of access: the bits of near ones."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    B, T, dt = 2, 21, torch.bfloat16
    c = make(B, T, hq, hk, D, R, "bf16", positions="each", seed=60)
    row = (hq + hk) * D + 16

    def far():
        base = torch.empty(2 ** 31 + T * row + 16, device=DEV, dtype=dt)
        part = lambda H, at: base.as_strided((B, T, H, D), (2 ** 31, row, D, 1), off + at) if H else None
        return part(hq, 0), part(hk, hq * D)

    want, grads = call(c, interleaved=interleaved), call_grad(c, interleaved=interleaved)
    check(c, want, 1e-5, interleaved)
    d = dict(c)
    d["q"], d["k"] = far()
    d["dyq"], d["dyk"] = far()
    for n in ("q", "k", "dyq", "dyk"):
        if c[n] is not None:
            d[n].copy_(c[n])
    got = call_grad(d, interleaved=interleaved, dq=d["dyq"], dk=d["dyk"])
    check_grad(c, got, 1e-5, interleaved)
    assert torch.equal(got[0], grads[0]) and (not hk or torch.equal(got[1], grads[1]))
    got = call(d, interleaved=interleaved, q_out=d["q"], k_out=d["k"])
    assert torch.equal(got[0], want[0]) and (not hk or torch.equal(got[1], want[1]))


def test_capture_and_replay_with_new_inputs():
    c = make(2, 64, 8, 2, 128, 128, "bf16", layout="fused", positions="each", seed=14)
    other = make(2, 64, 8, 2, 128, 128, "bf16", layout="fused", positions="each", seed=15)
    call(c), call_grad(c)
    torch.cuda.synchronize()
    ws = torch.empty(1 << 20, device=DEV, dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(c)
        grad = call_grad(c, workspace=ws)
    for src in (other, c):
        want = [t.clone() for t in call(src) + call_grad(src)]
        if src is other:
            c["q"]._base.copy_(other["q"]._base)
            for n in ("gq", "gk", "pos", "dyq", "dyk"):
                c[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out + grad, want):
            assert torch.equal(a, b)


def test_in_inference_mode_and_from_leaves():
    c = make(2, 5, 4, 2, 64, 64, "bf16", seed=19)
    want = call(c) + call_grad(c)
    with torch.inference_mode():
        got = call(c) + call_grad(c)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    d = {n: None if t is None else (t.requires_grad_() if t.is_floating_point() else t) for n, t in c.items()}
    got = call(d) + call_grad(d)
    for a, b in zip(got, want):
        assert not a.requires_grad and torch.equal(a, b)
    got[0].mul_(2)  # outputs are ordinary tensors, whatever they share
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0] * 2)


def test_two_streams_at_once():
    cs = [make(2, 300, 16, 4, 128, 128, "bf16", positions="each", seed=s) for s in (16, 17)]
    want = [call(c) + call_grad(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                got[i] = call(c) + call_grad(c)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_calls_close_behind_one_another():
    """Each call's input is the output of the one before it, on one stream."""
    c = make(1, 8, 32, 8, 128, 128, "bf16", seed=18)
    q, k = c["q"].clone(), c["k"].clone()
    for _ in range(20):
        call({**c, "q": q, "k": k}, q_out=q, k_out=k)
    torch.cuda.synchronize()
    p, r = c["q"].clone(), c["k"].clone()
    for _ in range(20):
        call({**c, "q": p, "k": r}, q_out=p, k_out=r)
        torch.cuda.synchronize()
    assert torch.equal(p, q) and torch.equal(r, k)


def test_binding_refusals():
    c = make(2, 5, 4, 2, 64, 64, "bf16", positions="each")
    x = c["q"]

    def bad(err, match=None, **kw):
        with pytest.raises(err, match=match):
            call({**c, **{k: v for k, v in kw.items() if k in c}}, **{k: v for k, v in kw.items() if k not in c})

    bad(TypeError, q=x.double())
    bad(ValueError, q=x[0, 0])
    bad(ValueError, q=x[..., ::2])
    bad(ValueError, k=c["k"][:, :4])
    bad(ValueError, k=c["k"][:1])
    bad(ValueError, k=c["k"].float())
    bad(ValueError, k=c["k"].cpu())
    bad(ValueError, match="need k", k=None)
    bad(ValueError, gq=c["gq"][:32])
    bad(TypeError, gq=c["gq"].float())
    bad(ValueError, match="together", sin=None)
    bad(ValueError, match="need cos", cos=None, sin=None)
    bad(ValueError, sin=c["sin"][:, :16])
    bad(ValueError, cos=torch.cat([c["cos"]] * 2, 1), sin=torch.cat([c["sin"]] * 2, 1))
    bad(TypeError, cos=c["cos"].half(), sin=c["sin"].half())
    bad(TypeError, cos=c["cos"].bfloat16())
    bad(ValueError, cos=c["cos"].cpu())
    bad(ValueError, match="rows", pos=None, cos=c["cos"][:4], sin=c["sin"][:4])
    bad(ValueError, pos=c["pos"][:, :4])
    bad(ValueError, pos=c["pos"][None])
    bad(TypeError, pos=c["pos"].float())
    bad(ValueError, pos=c["pos"].cpu())
    bad(ValueError, q_out=torch.empty_like(x)[:, :4])
    bad(nl.NormError, q_out=x[:, :1].expand(2, 5, 4, 64))
    bad(nl.NormError, q_out=torch.empty_like(x)[:, :, :1].expand(2, 5, 4, 64))
    bad(nl.NormError, k_out=c["q"][:, :, :2])
    with pytest.raises(nl.NormError):
        call(c, eps=0.0)
    wide = torch.zeros(2, 3, 4, 514, device=DEV)
    with pytest.raises(nl.NormError):
        nl.head_rms_rotary(wide)
    with pytest.raises(ValueError, match="together"):
        call_grad({**c, "dyk": None})
    with pytest.raises(ValueError):
        call_grad({**c, "dyq": c["dyq"][:, :, :2]})
    with pytest.raises(nl.NormError):
        call_grad(c, dq=c["q"])
    with pytest.raises(nl.NormError):
        call_grad(c, workspace=torch.empty(64, device=DEV))
    with pytest.raises(ValueError):
        call_grad(c, workspace=torch.empty(1 << 20))


def test_zz_no_device_errors():
    torch.cuda.synchronize()
    assert _lib.device_errors() == 0

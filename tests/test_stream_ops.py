"""The residual-stream operators on the CPU: the oracle against torch autograd
in 64 bits and central differences, and the C ABI's refusals (fake addresses;
every call is rejected, or has no rows, before it reaches the GPU)."""

import numpy as np
import pytest
import torch

import rmsnorm_ln_fwd_gb300 as nl
from oracle import stream_oracle as S
from rmsnorm_ln_fwd_gb300 import _build, _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2
I32, I64 = 0, 1
M = 0x100000  # fake, well-separated addresses: M, 2*M, ...


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def _inputs(N, H, B, seed=0):
    r = np.random.default_rng(seed)
    gate = None if B == 0 else r.normal(0.5, 0.5, (H,) if B == 1 else (B, H))
    return dict(x=r.normal(size=(N, H)), res=r.normal(size=(N, H)), gpost=r.normal(1, 0.2, H), gate=gate,
                gpre=r.normal(1, 0.2, H), dy=r.normal(size=(N, H)), dh=r.normal(size=(N, H)))


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("B", [0, 1, 3])
def test_oracle_gradient_is_autograd(B, post, pre):
    N, H, eps, alpha = 6, 10, 1e-5, 0.7
    c = _inputs(N, H, B)
    t = {k: None if v is None else torch.tensor(v, dtype=torch.float64, requires_grad=k not in ("dy", "dh"))
         for k, v in c.items()}
    p = t["x"]
    if post:
        p = p / torch.sqrt((p * p).mean(1, keepdim=True) + eps) * t["gpost"]
    if B:
        p = p * (t["gate"] if B == 1 else t["gate"].repeat_interleave(N // B, 0))
    h = alpha * t["res"] + p
    loss = (h * t["dh"]).sum()
    if pre:
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * t["gpre"]
        loss = loss + (y * t["dy"]).sum()
    loss.backward()
    fy, fh, rpost, rpre = S.sandwich_forward(c["x"], c["res"], c["gpost"] if post else None, c["gate"],
                                             c["gpre"] if pre else None, eps, alpha, post, pre)
    assert np.allclose(fh, h.detach().numpy(), rtol=1e-13, atol=1e-13)
    if pre:
        assert np.allclose(fy, y.detach().numpy(), rtol=1e-13, atol=1e-13)
    dx, dres, dgpost, dgate, dgpre = S.sandwich_backward(
        c["dy"] if pre else None, c["x"], fh if pre else None, rpost, rpre, c["gpost"] if post else None, c["gate"],
        c["gpre"] if pre else None, c["dh"], alpha)
    for got, name in ((dx, "x"), (dres, "res"), (dgpost, "gpost"), (dgate, "gate"), (dgpre, "gpre")):
        if got is None:
            assert t[name] is None or t[name].grad is None
        else:
            assert np.allclose(got, t[name].grad.numpy(), rtol=1e-11, atol=1e-12), name


def test_oracle_gradient_is_the_difference_quotient():
    N, H, eps, alpha, step = 4, 5, 1e-5, 0.7, 1e-6
    c = _inputs(N, H, 2, seed=3)

    def loss(**kw):
        d = {**c, **kw}
        y, h, _, _ = S.sandwich_forward(d["x"], d["res"], d["gpost"], d["gate"], d["gpre"], eps, alpha)
        return (y * c["dy"]).sum() + (h * c["dh"]).sum()

    _, h, rpost, rpre = S.sandwich_forward(c["x"], c["res"], c["gpost"], c["gate"], c["gpre"], eps, alpha)
    grads = S.sandwich_backward(c["dy"], c["x"], h, rpost, rpre, c["gpost"], c["gate"], c["gpre"], c["dh"], alpha)
    for name, g in zip(("x", "res", "gpost", "gate", "gpre"), grads):
        for i in np.ndindex(c[name].shape):
            up, down = c[name].copy(), c[name].copy()
            up[i] += step
            down[i] -= step
            # the quotient's own error: third derivatives of order 10 times step^2, rounding 1e-15 / step
            assert abs((loss(**{name: up}) - loss(**{name: down})) / (2 * step) - g[i]) < 1e-7


def test_oracle_lookup():
    r = np.random.default_rng(0)
    table, tokens = r.normal(size=(5, 4)), np.array([3, 0, 3, 7, -1])
    y, h, rstd = S.lookup_forward(tokens, table, 2.0, None, 1e-6)
    assert np.array_equal(h[0], 2 * table[3]) and not h[3].any() and not h[4].any()
    assert np.allclose((y[:3] ** 2).mean(1), 1, atol=1e-5)
    t = torch.tensor(table, requires_grad=True)
    dh = r.normal(size=(5, 4))
    (2.0 * t[torch.tensor([3, 0, 3])] * torch.tensor(dh[:3])).sum().backward()
    assert np.allclose(S.lookup_backward(dh, tokens, 5, 2.0), t.grad.numpy())
    assert not S.lookup_backward(dh, tokens, 5, 2.0, padding=3)[3].any()


# ------------------------------------------------------------------ refusals

def _join(lib, **kw):
    a = dict(x=M, ldx=64, r=2 * M, ldr=64, gpost=None, gate=None, ldg=64, B=0, gpre=None, y=3 * M, ldy=64, h=4 * M,
             ldh=64, rpost=None, rpre=None, N=4, H=64, eps=1e-6, alpha=1.0, norms=3, xd=BF16, wd=BF16, gd=BF16)
    a.update(kw)
    return lib.sandwich_rms(a["x"], a["ldx"], a["r"], a["ldr"], a["gpost"], a["gate"], a["ldg"], a["B"], a["gpre"],
                            a["y"], a["ldy"], a["h"], a["ldh"], a["rpost"], a["rpre"], a["N"], a["H"], a["eps"],
                            a["alpha"], a["norms"], a["xd"], a["wd"], a["gd"], None)


def test_join_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(x=None), dict(r=None), dict(h=None), dict(y=None), dict(H=0), dict(N=-1), dict(eps=0.0),
               dict(eps=nan), dict(alpha=nan), dict(alpha=inf), dict(norms=0), dict(norms=4), dict(ldx=63),
               dict(ldr=10), dict(ldy=63), dict(ldh=0), dict(y=M), dict(y=2 * M), dict(y=4 * M),
               dict(h=M + 2), dict(h=M, ldh=65), dict(r=M + 16, h=M),
               dict(gate=5 * M, B=3), dict(gate=5 * M, B=0), dict(gate=5 * M, B=-1), dict(gate=5 * M, B=8),
               dict(gate=5 * M, B=2, ldg=63), dict(gate=3 * M, B=1), dict(gate=4 * M + 4, B=1),
               dict(gpost=3 * M), dict(gpre=4 * M), dict(rpost=M), dict(rpre=3 * M), dict(rpost=5 * M, rpre=5 * M + 4),
               dict(gpre=5 * M, rpre=5 * M),
               # what belongs to a norm that is not taken
               dict(norms=2, gpost=5 * M), dict(norms=2, rpost=5 * M), dict(norms=1), dict(norms=1, y=None, gpre=5 * M),
               dict(norms=1, y=None, rpre=5 * M)):
        assert _join(lib, **kw) == INVALID, kw
    assert _join(lib, xd=7) == UNSUPPORTED
    assert _join(lib, xd=F32, wd=BF16) == UNSUPPORTED
    assert _join(lib, gate=5 * M, B=1, gd=F16) == UNSUPPORTED
    assert _join(lib, N=0, x=None, r=None, y=None, h=None) == OK
    assert _join(lib, N=0, gate=5 * M, B=2) == OK


def _grad(lib, **kw):
    a = dict(dy=M, lddy=64, x=2 * M, ldx=64, h=3 * M, ldh=64, rpost=4 * M, rpre=5 * M, gpost=None, gate=None, ldg=64,
             B=0, gpre=None, dh=6 * M, lddh=64, dx=7 * M, lddx=64, dr=8 * M, lddr=64, dgpost=None, dgate=None, lddg=64,
             dgpre=None, ws=9 * M, wsb=1 << 16, N=4, H=64, alpha=1.0, norms=3, xd=BF16, wd=BF16, gd=BF16)
    a.update(kw)
    return lib.sandwich_rms_grad(a["dy"], a["lddy"], a["x"], a["ldx"], a["h"], a["ldh"], a["rpost"], a["rpre"],
                                 a["gpost"], a["gate"], a["ldg"], a["B"], a["gpre"], a["dh"], a["lddh"], a["dx"],
                                 a["lddx"], a["dr"], a["lddr"], a["dgpost"], a["dgate"], a["lddg"], a["dgpre"],
                                 a["ws"], a["wsb"], a["N"], a["H"], a["alpha"], a["norms"], a["xd"], a["wd"],
                                 a["gd"], None)


def test_join_grad_refusals(lib):
    E = 10 * M
    for kw in (dict(dy=None), dict(x=None), dict(h=None), dict(rpost=None), dict(rpre=None), dict(dx=None),
               dict(dr=None), dict(H=0), dict(N=-1), dict(norms=0), dict(norms=8), dict(alpha=float("inf")),
               dict(ldx=63), dict(lddx=63), dict(lddh=1), dict(lddy=1), dict(ldh=1), dict(lddr=1),
               dict(dx=2 * M), dict(dx=3 * M), dict(dx=6 * M), dict(dx=M + 2), dict(dr=M), dict(dr=2 * M),
               dict(dr=3 * M), dict(dr=6 * M + 2), dict(dr=7 * M), dict(dx=4 * M), dict(dr=5 * M),
               dict(dgate=E), dict(gate=E, B=3), dict(gate=E, B=1, dgate=E + 2),
               dict(dgpost=E, dgpre=E + 64), dict(dgpre=7 * M), dict(dgpost=M), dict(dgpre=4 * M),
               dict(norms=1), dict(norms=2), dict(norms=1, dy=None, h=None, rpre=None, dh=None),
               dict(norms=2, rpost=None, dgpost=E), dict(norms=1, dy=None, h=None, rpre=None, dgpre=E)):
        assert _grad(lib, **kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=9 * M + 4), dict(ws=M), dict(ws=E), dict(ws=8 * M), dict(ws=4 * M)):
        assert _grad(lib, dgpre=E, **kw) == WORKSPACE, kw
    assert _grad(lib, xd=9) == UNSUPPORTED
    assert _grad(lib, gate=E, B=1, gd=F16) == UNSUPPORTED


def _look(lib, **kw):
    a = dict(t=M, ldt=64, V=10, k=2 * M, it=I64, g=None, y=3 * M, ldy=64, h=4 * M, ldh=64, rstd=None, N=4, H=64,
             eps=1e-6, scale=1.0, xd=BF16, wd=BF16)
    a.update(kw)
    return lib.embedding_rms(a["t"], a["ldt"], a["V"], a["k"], a["it"], a["g"], a["y"], a["ldy"], a["h"], a["ldh"],
                             a["rstd"], a["N"], a["H"], a["eps"], a["scale"], a["xd"], a["wd"], None)


def test_lookup_refusals(lib):
    for kw in (dict(t=None), dict(k=None), dict(h=None), dict(y=None), dict(V=0), dict(V=1 << 31), dict(H=0),
               dict(N=-1), dict(N=1 << 31), dict(eps=0.0), dict(scale=float("nan")), dict(ldt=63), dict(ldy=1),
               dict(ldh=1), dict(h=M), dict(y=4 * M), dict(y=2 * M), dict(g=3 * M), dict(rstd=2 * M), dict(rstd=4 * M)):
        assert _look(lib, **kw) == INVALID, kw
    assert _look(lib, it=2) == UNSUPPORTED
    assert _look(lib, xd=BF16, wd=F16) == UNSUPPORTED
    assert _look(lib, N=0, t=None, k=None, h=None, y=None) == OK
    plain = lambda **kw: lib.embedding_lookup(*({**dict(t=M, ldt=64, V=10, k=2 * M, it=I32, h=3 * M, ldh=64, N=4,  # noqa: E731
                                                        H=64, scale=1.0, xd=F32, s=None), **kw}.values()))
    assert plain(h=M + 4) == INVALID
    assert plain(scale=float("inf")) == INVALID
    assert plain(it=5) == UNSUPPORTED
    assert plain(N=0, t=None, k=None, h=None) == OK


def test_lookup_grad_refusals(lib):
    need = lib.embedding_grad_workspace_bytes(4, 64)
    assert need >= 2 * 4 * 8 + 2 * 64 * 4
    assert lib.embedding_grad_workspace_bytes(-1, 64) == 0
    assert lib.embedding_grad_workspace_bytes(4, 0) == 0
    assert lib.embedding_grad_workspace_bytes(0, 64) > 0

    def g(**kw):
        a = dict(dh=M, lddh=64, k=2 * M, it=I64, dt=3 * M, lddt=64, V=10, ws=4 * M, wsb=need, N=4, H=64, scale=1.0,
                 pad=-1, acc=0, xd=BF16, wd=BF16, s=None)
        a.update(kw)
        return lib.embedding_grad(*a.values())
    for kw in (dict(dh=None), dict(k=None), dict(dt=None), dict(V=0), dict(H=0), dict(N=-1), dict(pad=10),
               dict(pad=-2), dict(scale=float("nan")), dict(dh=M + 1), dict(dt=3 * M + 1), dict(k=2 * M + 4), dict(lddh=63), dict(lddt=63), dict(dt=M), dict(dt=2 * M)):
        assert g(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(wsb=need - 1), dict(ws=4 * M + 8), dict(ws=M), dict(ws=3 * M)):
        assert g(**kw) == WORKSPACE, kw
    assert g(it=3) == UNSUPPORTED
    assert g(xd=BF16, wd=F16) == UNSUPPORTED


@pytest.mark.parametrize("es,E", [(2, 16), (4, 8)])
def test_row_groups_stay_within_the_workspace(es, E):
    """The gradient's row groups a CTA (512 or 256 threads, whole warps for E
    columns a thread, at most eight) against the bound the workspace is sized
    by: transcriptions of both rules, every width."""
    for H in range(1, 20000):
        warps = (H + 511) // 512
        bound = 1 if warps >= 16 else min(8, 16 // warps)
        tpr = (H + 32 * E - 1) // (32 * E) * 32
        for threads in (256, 512):
            if tpr <= threads:
                assert min(threads // tpr, 8) <= bound


def test_pointers_between_elements_are_refused(lib):
    E = 10 * M
    for kw in (dict(x=M + 1), dict(r=2 * M + 1), dict(y=3 * M + 1), dict(h=4 * M + 1), dict(gpost=E + 1),
               dict(gpre=E + 1), dict(gate=E + 1, B=1), dict(rpost=E + 2), dict(rpre=E + 2),
               dict(gpre=E + 2, wd=F32), dict(gate=E + 2, B=1, gd=F32)):
        assert _join(lib, **kw) == INVALID, kw
    for kw in (dict(dy=M + 1), dict(x=2 * M + 1), dict(h=3 * M + 1), dict(rpost=4 * M + 2), dict(dh=6 * M + 1),
               dict(dx=7 * M + 1), dict(dr=8 * M + 1), dict(dgpre=E + 1), dict(gate=E, B=1, dgate=11 * M + 1)):
        assert _grad(lib, **kw) == INVALID, kw
    for kw in (dict(t=M + 1), dict(k=2 * M + 4), dict(k=2 * M + 2, it=I32), dict(y=3 * M + 1), dict(h=4 * M + 1),
               dict(g=5 * M + 1), dict(rstd=5 * M + 2)):
        assert _look(lib, **kw) == INVALID, kw


def test_host_tensors_are_refused():
    x, v = torch.zeros(4, 8), torch.ones(8)
    r = torch.ones(4)
    tok = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: nl.sandwich_rms(x, x), lambda: nl.sandwich_rms_grad(x, x, x, r, r, v, None, v),
                 lambda: nl.embedding_lookup(tok, x), lambda: nl.embedding_rms(tok, x),
                 lambda: nl.embedding_grad(x, tok, 4)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def _split(N, u, U):
    return N * u // U, N * (u + 1) // U


@pytest.mark.parametrize("N,U,run", [(12, 5, 4), (12, 5, 3), (12, 12, 12), (100, 7, 10), (100, 7, 50), (97, 8, 97),
                                     (60, 59, 2), (60, 1, 6), (1000, 304, 8), (30, 4, 1), (64, 3, 32)])
def test_run_partials_cover_every_run_once(N, U, run):
    """The index arithmetic of the gate gradient's partial rows: what the units
    leave and what the second kernel reads are the same slots, and every run is
    finished exactly once (a transcription of the kernels' rules)."""
    left, done = {}, []
    for u in range(U):
        lo, hi = _split(N, u, U)
        assert hi > lo
        first = lo // run
        for seg in range(first, (hi - 1) // run + 1):
            whole = seg * run >= lo and (seg + 1) * run <= hi
            rows = range(max(lo, seg * run), min(hi, (seg + 1) * run))
            if whole:
                done.append((seg, list(rows)))
            else:
                slot = 2 * u + (0 if seg == first else 1)
                assert slot not in left
                left[slot] = list(rows)

    def unit_of(r):
        return ((r + 1) * U - 1) // N

    runs = N // run
    by_boundary = runs > U - 1
    read = []
    if run > 1 and U > 1:
        for k in range(U - 1 if by_boundary else runs):
            seg = k
            if by_boundary:
                r = N * (k + 1) // U
                if r % run == 0:
                    continue
                seg = r // run
                if unit_of(seg * run) != k:
                    continue
            u0, u1 = unit_of(seg * run), unit_of((seg + 1) * run - 1)
            if u0 == u1:
                continue
            slots = [2 * u0 + (0 if (N * u0 // U) // run == seg else 1)] + [2 * u for u in range(u0 + 1, u1 + 1)]
            read += slots
            done.append((seg, sum((left[s] for s in slots), [])))
    assert sorted(read) == sorted(left)
    assert sorted(done) == [(s, list(range(s * run, (s + 1) * run))) for s in range(runs)]


@pytest.mark.parametrize("tokens", [[0], [1] * 33, list(range(70)), [2] * 32 + [3] * 32 + [4] * 40, [5, 5] + [7] * 200,
                                    [9] * 64, [1] * 31 + [2] * 2 + [3] * 31])
def test_tile_partials_cover_every_token_once(tokens):
    """The same for the table's gradient: tiles of 32 sorted tokens."""
    K, n = 32, len(tokens)
    tiles = (n + K - 1) // K
    partial, done = {}, {}
    for t in range(tiles):
        ids = tokens[t * K:(t + 1) * K]
        before = tokens[t * K - 1] if t else None
        after = tokens[(t + 1) * K] if (t + 1) * K < n else None
        got = []
        for i, v in enumerate(ids):
            got.append(t * K + i)
            if i + 1 < len(ids) and ids[i + 1] == v:
                continue
            if before == ids[0] and v == ids[0]:
                partial[2 * t] = got
            elif i + 1 == len(ids) and after == v:
                partial[2 * t + 1] = got
            else:
                assert v not in done
                done[v] = got
            got = []
    used = []
    for b in range(tiles - 1):
        end = (b + 1) * K
        v = tokens[end]
        if tokens[end - 1] != v or (b > 0 and tokens[b * K - 1] == v):
            continue
        got, t = list(partial[2 * b + 1]), b + 1
        used.append(2 * b + 1)
        while t * K < n and tokens[t * K] == v:
            got += partial[2 * t]
            used.append(2 * t)
            t += 1
        assert v not in done
        done[v] = got
    assert sorted(used) == sorted(partial)
    assert done == {v: [i for i, w in enumerate(tokens) if w == v] for v in set(tokens)}


# ------------------------------------------------------------------ the binding's row views

def _row_view(t):
    _build.build()
    return _lib.bind().row_view(t)


@pytest.mark.parametrize("shape,strides", [((5, 8), (8, 1)), ((5, 8), (11, 1)), ((2, 3, 8), (24, 8, 1)),
                                           ((2, 3, 8), (30, 10, 1)), ((2, 1, 3, 8), (24, 7, 8, 1)), ((1, 8), (0, 1)),
                                           ((4, 1, 8), (9, 0, 1)), ((1, 3, 8), (0, 8, 1)), ((3, 1), (5, 77)),
                                           ((2, 3, 4, 8), (120, 40, 10, 1)), ((8,), (1,))])
def test_row_views(shape, strides):
    """Row r of the view is the r-th row of the tensor, in order."""
    t = torch.arange(1000.0).as_strided(shape, strides)
    N, H, ld = _row_view(t)
    assert torch.equal(torch.arange(1000.0).as_strided((N, H), (ld, 1)), t.reshape(N, H))


@pytest.mark.parametrize("shape,strides", [
    ((4, 6, 8), (8, 0, 1)),        # a row for each sequence, over its tokens: the gradient of y.sum(1)
    ((4, 6, 8), (0, 8, 1)),        # over the sequences
    ((4, 3, 6, 8), (24, 8, 0, 1)), ((4, 3, 6, 8), (8, 0, 0, 1)), ((4, 3, 6, 8), (8, 0, 8, 1)), ((4, 3, 6, 8), (0, 8, 0, 1)),
    ((4, 1, 6, 8), (8, 8, 0, 1)), ((4, 6, 1, 8), (8, 0, 8, 1)),
    ((4, 6, 8), (8, 32, 1)), ((4, 6, 8), (50, 8, 1)), ((4, 6, 8), (48, 8, 2)), ((4, 6, 8), (1, 8, 1))])
def test_row_views_that_do_not_flatten(shape, strides):
    with pytest.raises(ValueError, match="flatten|contiguous"):
        _row_view(torch.zeros(2000).as_strided(shape, strides))


@pytest.mark.parametrize("shape", [(6, 8), (4, 6, 8), (2, 3, 6, 8)])
def test_row_views_of_one_expanded_row(shape, lib):
    """One row for all: a row stride of 0, which the library refuses."""
    t = torch.zeros(8).expand(shape)
    N, H, ld = _row_view(t)
    assert ld == 0 and N * H == t.numel()
    assert _join(lib, N=N, H=H, ldx=ld) == _join(lib, N=N, H=H, ldr=ld) == _join(lib, N=N, H=H, ldh=ld) == INVALID
    assert _grad(lib, N=N, H=H, lddy=ld) == _grad(lib, N=N, H=H, lddh=ld) == _grad(lib, N=N, H=H, lddx=ld) == INVALID


@pytest.mark.parametrize("H", [1, 64, 4096])
def test_lookup_grad_workspace_grows_with_the_tokens(lib, H):
    """A workspace for a batch serves every smaller one: short tiles for few
    tokens must not ask for more than long tiles for many."""
    sizes = [lib.embedding_grad_workspace_bytes(n, H)
             for n in [0, 1, 7, 8, 9, *range(4080, 4120), 6000, *range(8180, 8210), 16384, 16385, 20000, 1 << 20]]
    assert sizes == sorted(sizes)
    # what a call needs at least: two buffers of pairs, and two partial rows and an owner a tile
    for n, tile in ((4096, 8), (4097, 16), (8192, 16), (8193, 32), (100000, 32)):
        tiles = -(-n // tile)
        assert lib.embedding_grad_workspace_bytes(n, H) >= 16 * n + 8 * (1 + tiles) + 8 * tiles * H


def test_a_binding_for_another_pytorch_is_not_loaded(tmp_path, monkeypatch):
    _build.build()
    with open(_build.BIND, "rb") as f:
        built = f.read()
    mark = b"norm_bind_torch=" + torch.__version__.encode()
    assert built.count(mark) == 1 and _build.bind_torch() == torch.__version__ and _build.bind_up_to_date()
    other = tmp_path / "_bind.so"
    other.write_bytes(built.replace(mark, mark[:-1] + b"?"))
    monkeypatch.setattr(_build, "BIND", str(other))
    monkeypatch.setattr(_lib, "_bind", None)
    assert not _build.bind_up_to_date()
    with pytest.raises(RuntimeError, match="built for PyTorch"):
        _lib.bind()

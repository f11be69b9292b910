"""The gated delta rule with one decay per head and the drafts' verification: what the entry points
refuse, on the host (CPU only: no call here reaches a kernel launch), and the fp64 reference's gradients
against differences."""
import ctypes
import os

import numpy as np
import pytest

import gated_delta_rule_78_amd as kda
import gdr_ref as ref

OK, NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUP, WORKSPACE = 0, -1, -2, -3, -4, -5, -6, -8
BASE, MB = 1 << 40, 1 << 20
NUL = ctypes.c_void_p(None)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        pytest.skip("libkda.so not built")
    return kda.lib()


def _p(i, off=0):  # never dereferenced: every call below is refused before a launch
    return ctypes.c_void_p(BASE + i * 64 * MB + off)


def _fwd(L, B=1, T=64, H=2, Hk=2, dk=64, dv=64, chunk=64, dtype=0, s0=None, sT=None, ws=None, nws=None, varlen=None,
         cu=None, **kw):
    sh = kda.Shape(B, T, H, dk, dv, chunk, dtype)
    a = dict(q=_p(0), k=_p(1), v=_p(2), g=_p(3), b=_p(4), o=_p(5))
    a.update(kw)
    tail = (a["q"], a["k"], a["v"], a["g"], a["b"], s0, a["o"], sT, _p(20) if ws is None else ws,
            ctypes.c_size_t(1 << 40 if nws is None else nws), None)
    if varlen is not None:
        return L.kda_gdr_chunk_fwd_varlen(ctypes.byref(sh), Hk, cu, varlen, *tail)
    return L.kda_gdr_chunk_fwd(ctypes.byref(sh), Hk, *tail)


def _bwd(L, B=1, T=64, H=2, Hk=2, dk=64, dv=64, chunk=64, dtype=0, ws=None, nws=None, varlen=None, cu=None, **kw):
    sh = kda.Shape(B, T, H, dk, dv, chunk, dtype)
    a = dict(q=_p(0), k=_p(1), v=_p(2), g=_p(3), b=_p(4), s0=_p(5), d_o=_p(6), dsT=_p(7), dq=_p(8), dk_=_p(9),
             dv_=_p(10), dg=_p(11), db=_p(12), ds0=_p(13))
    a.update(kw)
    tail = (a["q"], a["k"], a["v"], a["g"], a["b"], a["s0"], a["d_o"], a["dsT"], a["dq"], a["dk_"], a["dv_"], a["dg"],
            a["db"], a["ds0"], _p(20) if ws is None else ws, ctypes.c_size_t(1 << 40 if nws is None else nws), None)
    if varlen is not None:
        return L.kda_gdr_chunk_bwd_varlen(ctypes.byref(sh), Hk, cu, varlen, *tail)
    return L.kda_gdr_chunk_bwd(ctypes.byref(sh), Hk, *tail)


def _dec(L, tokens=False, B=1, T=1, H=2, Hk=2, dk=64, dv=64, dtype=0, counts=None, update=1, **kw):
    sh = kda.Shape(B, T, H, dk, dv, 0, dtype)
    a = dict(q=_p(0), k=_p(1), v=_p(2), g=_p(3), b=_p(4), S=_p(6), o=_p(7))
    a.update(kw)
    tail = (a["q"], a["k"], a["v"], a["g"], a["b"], a["S"], a["o"], None)
    if tokens:
        return L.kda_gdr_decode_tokens(ctypes.byref(sh), Hk, counts, update, *tail)
    return L.kda_gdr_decode_step(ctypes.byref(sh), Hk, *tail)


def _tok(L, **k):
    return _dec(L, tokens=True, **k)


@pytest.mark.parametrize("f", [_fwd, _bwd, _dec, _tok])
def test_refuses_shapes(L, f):
    assert f(L, dtype=7) == DTYPE
    assert f(L, H=0, Hk=1) == SHAPE and f(L, B=-1) == SHAPE and f(L, Hk=0) == SHAPE
    assert f(L, H=4, Hk=3) == SHAPE and f(L, H=2, Hk=4) == SHAPE and f(L, H=65536, Hk=65536) == SHAPE
    assert f(L, dk=96) == UNSUP and f(L, dv=32) == UNSUP
    for name in ("q", "k", "v", "g", "b"):
        assert f(L, **{name: NUL}) == NULL, name


def test_refuses_sizes(L):
    assert _fwd(L, T=-1) == SHAPE and _bwd(L, T=-1) == SHAPE and _tok(L, T=-1) == SHAPE
    assert _fwd(L, B=1 << 16, T=1 << 16, H=2) == SHAPE
    assert _fwd(L, chunk=32) == UNSUP and _bwd(L, chunk=32) == UNSUP
    # a launch counts its threads in 32 bits
    n = 1 << 23
    assert _fwd(L, T=64, varlen=n, cu=_p(14)) == SHAPE and _bwd(L, T=64, varlen=n, cu=_p(14)) == SHAPE
    assert _fwd(L, B=1 << 23, T=1, H=1, Hk=1) == SHAPE and _bwd(L, B=1 << 23, T=1, H=1, Hk=1) == SHAPE
    assert _dec(L, B=1 << 20, H=8, Hk=8, dv=128) == SHAPE


def test_refuses_alignment(L):
    for name in ("q", "k", "v", "o"):
        assert _fwd(L, **{name: _p(14, 8)}) == ALIGN
    assert _fwd(L, g=_p(14, 2)) == ALIGN and _fwd(L, b=_p(14, 1)) == ALIGN and _fwd(L, b=_p(14, 2), dtype=1) == ALIGN
    assert _fwd(L, s0=_p(14, 4)) == ALIGN and _fwd(L, sT=_p(14, 4)) == ALIGN and _fwd(L, ws=_p(14, 16)) == ALIGN
    for name in ("q", "k", "v", "d_o", "dq", "dk_", "dv_", "s0", "dsT", "ds0"):
        assert _bwd(L, **{name: _p(14, 8)}) == ALIGN, name
    assert _bwd(L, dg=_p(14, 2)) == ALIGN and _bwd(L, db=_p(14, 1)) == ALIGN and _bwd(L, ws=_p(14, 16)) == ALIGN
    assert _dec(L, S=_p(14, 8)) == ALIGN and _dec(L, q=_p(14, 1)) == ALIGN and _dec(L, g=_p(14, 2)) == ALIGN
    assert _tok(L, counts=_p(14, 2)) == ALIGN


def test_refuses_overlap(L):
    for x in range(5):
        assert _fwd(L, o=_p(x)) == ALIAS and _fwd(L, sT=_p(x)) == ALIAS and _fwd(L, ws=_p(x)) == ALIAS
        assert _dec(L, o=_p(x)) == ALIAS and _dec(L, S=_p(x)) == ALIAS
    assert _fwd(L, s0=_p(14), sT=_p(14, 256)) == ALIAS and _dec(L, o=_p(6)) == ALIAS
    assert _tok(L, counts=_p(6)) == ALIAS and _tok(L, counts=_p(7)) == ALIAS
    for out in ("dq", "dk_", "dv_", "dg", "db", "ds0"):
        for x in range(8):
            assert _bwd(L, **{out: _p(x)}) == ALIAS, (out, x)
    assert _bwd(L, dq=_p(9)) == ALIAS and _bwd(L, dg=_p(12)) == ALIAS and _bwd(L, ws=_p(8)) == ALIAS


def test_refuses_decode_without_a_purpose(L):
    assert _tok(L, q=NUL) == NULL and _tok(L, o=NUL) == NULL   # outputs need both
    assert _tok(L, q=NUL, o=NUL, update=0) == OK               # nothing to do: no launch
    assert _tok(L, T=0) == OK and _tok(L, B=0) == OK


def test_workspaces(L):
    sh = lambda **k: ctypes.byref(kda.Shape(*[dict(dict(B=1, T=64, H=2, dk=64, dv=64, chunk=64, dtype=0), **k)[n]
                                              for n in ("B", "T", "H", "dk", "dv", "chunk", "dtype")]))
    f, b = L.kda_gdr_chunk_fwd_workspace_size, L.kda_gdr_chunk_bwd_workspace_size
    n = f(sh())
    assert n > 0 and _fwd(L, nws=n - 1) == WORKSPACE and _fwd(L, ws=NUL) == NULL
    m = b(sh())
    assert m > n and _bwd(L, nws=m - 1) == WORKSPACE and _bwd(L, ws=NUL) == NULL
    for bad in (dict(dk=96), dict(T=-1), dict(dtype=5), dict(B=-1)):
        assert f(sh(**bad)) == 0 and b(sh(**bad)) == 0
    fv, bv = L.kda_gdr_chunk_fwd_varlen_workspace_size, L.kda_gdr_chunk_bwd_varlen_workspace_size
    n = fv(sh(), 3)
    assert n > 0 and fv(sh(), -1) == 0 and bv(sh(), -1) == 0 and fv(sh(B=2), 3) == 0
    assert _fwd(L, varlen=3, cu=_p(14), nws=n - 1) == WORKSPACE
    assert _bwd(L, varlen=3, cu=_p(14), nws=bv(sh(), 3) - 1) == WORKSPACE


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,n", [(131072, 1024), (131072, 16384), (5000, 5000), (0, 4096)])
def test_packed_workspaces(L, T, n, dtype):
    """A further sequence takes at most one chunk's triangles and decays (and in the backward its two states), a list entry
    and its decay gradient's sums; no state of segments."""
    H, d, es = 32, 128, (2, 4)[dtype]
    sh = ctypes.byref(kda.Shape(1, T, H, d, d, 64, dtype))
    chunks, state = T // 64 + n, H * d * d * 4
    tri = chunks * H * (2560 + 98)  # two triangles, and decays and strengths, in pairs of fp32
    ends = T // (64 * 8) * state
    assert L.kda_gdr_chunk_fwd_varlen_workspace_size(sh, n) <= tri * 8 + 3 * ends + 32 * n + T + 65536
    rows = T * H * (d * es + 3 * 4 * (d // 64))
    keep = T // (64 * (8, 4)[dtype]) * state
    assert (L.kda_gdr_chunk_bwd_varlen_workspace_size(sh, n)
            <= tri * 8 + 3 * ends + chunks * H * d * d * es * 2 + keep + rows + n * H * 64 + T * H + 65536)


def test_packed_refusals(L):
    for f in (_fwd, _bwd):
        assert f(L, varlen=3, cu=None) == NULL
        assert f(L, varlen=-1, cu=_p(14)) == SHAPE
        assert f(L, B=2, varlen=3, cu=_p(14)) == SHAPE
        assert f(L, varlen=3, cu=_p(14, 2)) == ALIGN
    assert _fwd(L, varlen=3, cu=_p(5)) == ALIAS and _bwd(L, varlen=3, cu=_p(8)) == ALIAS


def _ver(L, B=2, K=3, V=100, dtype=1, nws=1 << 30, **kw):
    a = dict(p=_p(0), x=_p(1), q=_p(2), u=_p(3), ul=_p(4), n=_p(5), t=_p(6), ws=_p(7))
    a.update(kw)
    return L.kda_verify_drafts(B, K, V, dtype, a["p"], a["x"], a["q"], a["u"], a["ul"], a["n"], a["t"], a["ws"],
                               ctypes.c_size_t(nws), None)


def test_verify_refuses(L):
    assert _ver(L, dtype=2) == DTYPE
    assert _ver(L, B=-1) == SHAPE and _ver(L, K=-1) == SHAPE and _ver(L, V=0) == SHAPE and _ver(L, V=(1 << 30) + 1) == SHAPE
    assert _ver(L, B=1 << 25, K=1) == SHAPE and _ver(L, B=1 << 20, V=1 << 20) == SHAPE
    assert _ver(L, B=1 << 20, K=1 << 12, V=1) == SHAPE
    for nm in ("p", "x", "u", "ul", "n", "t", "ws"):
        assert _ver(L, **{nm: NUL}) == NULL, nm
    for nm in ("p", "x", "q", "u", "ul", "n", "t", "ws"):
        assert _ver(L, **{nm: _p(9, 2)}) == ALIGN, nm
    assert _ver(L, dtype=0, p=_p(9, 1)) == ALIGN and _ver(L, ws=_p(9, 4)) == ALIGN
    size = L.kda_verify_drafts_workspace_size
    assert _ver(L, nws=size(2, 3, 100, 1) - 1) == WORKSPACE
    assert size(2, 3, 0, 1) == 0 and size(2, 3, 100, 9) == 0
    for out in ("n", "t", "ws"):
        for x in range(5):
            assert _ver(L, **{out: _p(x)}) == ALIAS, (out, x)
    assert _ver(L, n=_p(6)) == ALIAS and _ver(L, t=_p(7)) == ALIAS
    assert _ver(L, B=0) == OK


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    q, k, v, g, b = z(1, 8, 2, 64), z(1, 8, 2, 64), z(1, 8, 4, 64), z(1, 8, 4), z(1, 8, 4)
    f = kda.gdr_chunk_fwd
    for args in ((q.bfloat16(), k, v, g, b), (q, k, v.bfloat16(), g, b), (q, k, v, g.bfloat16(), b), (q, k, v, g, b.bfloat16()),
                 (q.half(), k.half(), v.half(), g, b.half())):
        with pytest.raises(TypeError):
            f(*args)
    for args in ((q, k, v, z(4), b), (q, k, v, g, z(1, 8, 2)), (q, k, z(1, 8, 3, 64), z(1, 8, 3), z(1, 8, 3)),
                 (z(1, 8, 2, 128), k, v, g, b), (q, k, z(1, 9, 4, 64), g, b)):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(ValueError):
        f(q, k, v, g, b, initial_state=z(1, 2, 64, 64))
    with pytest.raises(ValueError):
        f(*(torch.cat([x, x]) for x in (q, k, v, g, b)), cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(TypeError):
        f(q, k, v, g, b, cu_seqlens=torch.tensor([0, 8]))
    with pytest.raises(ValueError):
        kda.gdr_chunk_bwd(q, k, v, g, b, z(1, 8, 2, 64))
    with pytest.raises(ValueError):  # no CPU fallback
        f(q, k, v, g, b)
    one = [x[:, 0] for x in (q, k, v, g, b)]
    with pytest.raises(ValueError):
        kda.gdr_decode_step(*one, z(1, 2, 64, 64))
    with pytest.raises(ValueError):
        kda.gdr_decode_step(*one, z(1, 4, 64, 64))
    S, d = z(1, 4, 64, 64), kda.gdr_decode_tokens
    with pytest.raises(ValueError):
        d(*one, S)
    with pytest.raises(ValueError):
        d(None, k, v, g, b, S, update=False)
    with pytest.raises(ValueError):
        d(None, k, v, g, b, S, out=z(1, 8, 4, 64))
    with pytest.raises(ValueError):
        d(None, k, v, g, b, S, qk_prep=dict(norm="l2"))
    for bad in (torch.tensor([3]), torch.tensor([3, 3], dtype=torch.int32)):
        with pytest.raises(TypeError):
            d(q, k, v, g, b, S, counts=bad)
    p, x, pq, u, ul = z(2, 4, 9), z(2, 3, dt=torch.int32), z(2, 3, 9), z(2, 3), z(2)
    ver = kda.verify_drafts
    for args in ((p, x.long(), pq, u, ul), (p, x, pq, u.double(), ul), (p.half(), x, pq.half(), u, ul)):
        with pytest.raises(TypeError):
            ver(*args)
    for args in ((z(2, 3, 9), x, pq, u, ul), (p, x, z(2, 3, 8), u, ul), (p, x, pq.bfloat16(), u, ul), (p, x, pq, z(2, 4), ul),
                 (p, x, pq, u, z(3)), (z(2, 4, 0), x, z(2, 3, 0), u, ul), (p, x, pq, u, ul)):
        with pytest.raises(ValueError):
            ver(*args)


@pytest.mark.parametrize("seed", [0, 1])
def test_reference_gradient_against_differences(seed):
    """The reference's gradients against central differences of its own loss, in fp64: with a step of 1e-5 on
    values of order one, truncation (1e-10) and cancellation (1e-16 / 1e-5) stay under 1e-8 of the loss's scale."""
    r = np.random.default_rng(seed)
    B, T, Hk, H, dk, dv = 2, 9, 2, 4, 5, 3
    x = [r.standard_normal(s) for s in ((B, T, Hk, dk), (B, T, Hk, dk), (B, T, H, dv), (B, T, H), (B, T, H), (B, H, dk, dv))]
    x[1] /= np.linalg.norm(x[1], axis=-1, keepdims=True)
    x[3], x[4] = -0.5 * np.abs(x[3]), 2.0 / (1.0 + np.exp(-x[4]))
    u, w = r.standard_normal((B, T, H, dv)), r.standard_normal((B, H, dk, dv))

    def loss(*a):
        o, sT = ref.gdr_fwd(*a)
        return (o * u).sum() + (sT * w).sum()

    grads = ref.gdr_bwd(*x[:5], u, x[5], w)
    for i, gr in enumerate(grads):
        d, h = r.standard_normal(x[i].shape), 1e-5
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + h * d, x[i] - h * d
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        assert abs(num - (gr * d).sum()) <= 1e-7 * (1 + np.abs(gr * d).sum()), i


def test_verified_tokens_are_distributed_as_the_target():
    """The reference's rule on a grid of random numbers: the token that comes out has the target's probabilities,
    whatever the draft's.  One draft, a grid of n x n numbers: off by at most a few cells of 1 / n for each token."""
    V, n = 5, 200
    r = np.random.default_rng(2)
    p, q = r.dirichlet(np.ones(V), 2), r.dirichlet(np.ones(V))
    got = np.zeros(V)
    grid = (np.arange(n) + 0.5) / n
    for x in range(V):
        # of the draft x: a share of min(1, p / q) stands, the rest is drawn from max(p - q, 0)
        share = np.mean(grid * q[x] < p[0, x])
        got[x] += q[x] * share
        if share < 1:
            one = lambda ul: ref.verify(p[None], np.array([[x]]), q[None, None], np.array([[1 - 1e-9]]), np.array([ul]))[1][0]
            tokens = np.bincount([one(ul) for ul in grid], minlength=V) / n
            got += q[x] * (1 - share) * tokens
    assert np.abs(got - p[0]).max() <= 3.0 / n


def test_verify_refuses_counts_that_pass_their_types(L):
    """K + 1 behind 32 bits, and probabilities whose bytes pass 64."""
    size = L.kda_verify_drafts_workspace_size
    for B, K, V in ((1, 2 ** 31 - 1, 100), (64, 2 ** 31 - 1, 100), (1, (1 << 30) + 1, 1), (32, (1 << 26) - 1, 1 << 30),
                    (1, 1 << 30, 1 << 30)):
        for dtype in (0, 1):
            assert size(B, K, V, dtype) == 0 and _ver(L, B=B, K=K, V=V, dtype=dtype) == SHAPE, (B, K, V)
    # the largest that are left, up to the workspace's check
    assert size(1, 1 << 30, 100, 1) > 0 and _ver(L, B=1, K=1 << 30, V=100, nws=0) == WORKSPACE
    assert size(31, (1 << 24) - 1, 1 << 30, 0) > 0


@pytest.mark.parametrize("B,T,H", [(1 << 30, 1 << 30, 16), (1 << 30, 1 << 30, 32768), (2 ** 31 - 1, 2 ** 31 - 1, 48)])
def test_row_counts_that_pass_64_bits(L, B, T, H):
    """B T H beyond 64 bits (2^64, 2^75; 48 (2^31 - 1)^2) is refused like any other count of rows over 2^32."""
    ref_ = ctypes.byref(kda.Shape(B, T, H, 64, 64, 64, 0))
    for size in (L.kda_gdr_chunk_fwd_workspace_size, L.kda_gdr_chunk_bwd_workspace_size, L.kda_lina_chunk_fwd_workspace_size):
        assert size(ref_) == 0
    assert L.kda_lina_chunk_bwd_workspace_size(ref_, H) == 0
    assert L.kda_chunk_fwd_workspace_size(ref_) == 0 and L.kda_chunk_bwd_workspace_size(ref_) == 0
    assert _fwd(L, B=B, T=T, H=H, Hk=H) == SHAPE and _bwd(L, B=B, T=T, H=H, Hk=H) == SHAPE
    assert _tok(L, B=B, T=T, H=H, Hk=H) == SHAPE

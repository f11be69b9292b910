"""The gated delta rule with one decay per head on the GPU against fp64 references (gpu).

Bounds, for each (batch, head) by itself.  With unit k and beta in [0, 2] a token's transition is not
expansive, so that an error once made in a state does not grow; what is left is what each chunk of 64
tokens adds.
 - fp32 results (fp32 inputs; states, their gradients and decay gradients of any inputs: three bf16 terms hold 24
   bits): a chunk's result passes four products one after another (K S, the triangular inverse, what it
   multiplies, K^T .), each a sum of at most 128 terms, off by about sqrt(128) 2^-24 of its terms' norm where roundings
   are independent; chunks add as independent errors do:  |err|_2 <= 4 sqrt(128) 2^-24 sqrt(1 + chunks) |x|_2, the
   norms over a head's tokens.  Scale floors where a result nearly cancels: its terms' norm.
   Decay gradients are carried over up to 512 tokens by differences of do . o and dv . v, which are larger than they
   are: the same on the norm of these.
 - bf16 outputs: a rounding is off by at most half a step, 2^-8 of the value, 2^-8 / sqrt(3) in the root mean
   square.  o takes its own, elementwise 2^-8 of the value, and two terms of what it is made from (2^-16 of them, in
   _out).  dv takes only its own: 2^-8 of the value and fp32's bound.  dq and dk take eight (their own, the two states', r's, u's,
   y's and the scores'): sqrt(8) 2^-8 / sqrt(3) of their terms' norm; held to 2^-6 of the result's, and where keys are
   equal, and terms cancel, of the terms' (_terms).  d_beta = sum_c z_c r_c takes one of each r_c (at most 2^-8 |z_c r_c|,
   z is fp32) and its own, elementwise: 2^-8 (|d_beta| + sum_c |z_c r_c|) (1 + 2^-6) and fp32's bound.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import gdr_ref as ref

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def _inputs(B, T, Hk, H, dk, dv, dtype, seed=0, beta=1.0, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)
    q, k, v, do = (unit(rn(B, T, Hk, dk)).to(dt), unit(rn(B, T, Hk, dk)).to(dt), rn(B, T, H, dv).to(dt),
                   rn(B, T, H, dv).to(dt))
    gl = -scale * torch.logspace(-2.5, 0.3, H) * torch.nn.functional.softplus(rn(B, T, H))
    b = (beta * torch.sigmoid(rn(B, T, H))).to(dt)
    return q, k, v, gl.float(), b, do


def _np(x):
    return None if x is None else x.detach().double().cpu().numpy()


def _dev(*xs):
    return [None if x is None else x.cuda().contiguous() for x in xs]


def _fp32(T, reach=1):
    """reach: where keys are equal and beta is 2, N = (I + A diag(beta))^-1 has entries of size 2 (1.008 ** 64 times that
    for keys whose squared length is 1.004 after a rounding to bf16) all over its triangle, and an error d of a score moves N by
    N d N: a sum over up to 64 tokens on either side, sqrt(64 . 64 / 2) 3.3 / 2 = 75 times as large; 64 of
    independent ones."""
    return reach * 4 * np.sqrt(128.0) * 2.0 ** -24 * np.sqrt(2.0 + T / 64)


def _norm(x, axes):
    return np.sqrt((x * x).sum(axes))


def _rel(x, r, bound, what, floor=0.0, axes=(1, 3)):
    """2-norms of each (batch, head): [B,T,H,.] with axes (1, 3), states [B,H,.,.] with (2, 3)."""
    x = _np(x)
    assert x.shape == r.shape and np.isfinite(x).all(), what
    err, ok = _norm(x - r, axes), bound * (_norm(r, axes) + floor) + 1e-30
    assert (err <= ok).all(), (what, (err / ok).max())


def _elem(x, r, fp, what):  # rounded once: dv
    x = _np(x)
    slack = fp * (np.sqrt((r * r).mean((1, 3), keepdims=True)) * 8 + np.abs(r))
    assert (np.abs(x - r) <= 2.0 ** -8 * np.abs(r) + slack).all(), what


def _out(o, r, rs, dtype, T, what="o", reach=1):
    """A head's outputs; v and the states are of order one, so that sqrt(T) is the norm of their terms."""
    scale = np.sqrt(T) + np.linalg.norm(rs)
    if dtype == "f32":
        return _rel(o, r, _fp32(T, reach), what, 0.1 * scale)
    x = _np(o)
    assert x.shape == r.shape and np.isfinite(x).all(), what
    # over 2^-8 of the value: what two terms leave, 2^-16 of three products' terms
    over = np.maximum(np.abs(x - r) - 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(r), 0.0)
    assert (_norm(over, (1, 3)) <= (3 * 2.0 ** -16 + _fp32(T, reach)) * (_norm(r, (1, 3)) + scale)).all(), what


def _check_fwd(B, T, Hk, H, dk, dv, dtype, s0=True, seed=0, beta=1.0, ins=None, reach=1):
    import torch

    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, _ = _inputs(B, T, Hk, H, dk, dv, dtype, seed, beta) if ins is None else ins
    S0 = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(seed + 1)) if s0 else None
    o, sT = kda.gdr_chunk_fwd(*_dev(q, k, v, g, b), initial_state=_dev(S0)[0])
    torch.cuda.synchronize()
    r, rs = ref.gdr_fwd(*(_np(x) for x in (q, k, v, g, b)), _np(S0))
    _out(o, r, rs, dtype, T, reach=reach)
    _rel(sT, rs, _fp32(T, reach), "final state", 1.0, (2, 3))
    return o, sT


def _check_bwd(B, T, Hk, H, dk, dv, dtype, s0=True, seed=0, beta=1.0, ins=None, cancels=False, reach=1):
    import torch

    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, do = _inputs(B, T, Hk, H, dk, dv, dtype, seed, beta) if ins is None else ins
    gen = torch.Generator().manual_seed(seed + 1)
    S0, dS = (torch.randn(B, H, dk, dv, generator=gen) for _ in range(2)) if s0 else (None, None)
    out = kda.gdr_chunk_bwd(*_dev(q, k, v, g, b, do), initial_state=_dev(S0)[0], d_final_state=_dev(dS)[0])
    torch.cuda.synchronize()
    _check_grads(out, (q, k, v, g, b, do), dtype, T, _np(S0), _np(dS), cancels, reach)
    return out


def _terms(q, k, v, g, b, do, S0, r):
    """Norms over a head's tokens of what dq and dk are sums of, for unit q and k: with u the rows that enter the state,
    y = dv, |do_i| (sum_j u_j^2 + |S|^2)^(1/2), and for dk |u_i| (sum_j do_j^2 + y_j^2)^(1/2) beside
    |y_i| (sum_j u_j^2 + |S|^2)^(1/2); j over the chunk, |S| the largest state's (a sum of u and S_0 itself)."""
    # u_t = (S_t - e^g S_{t-1})^T k_t / |k|^2: from the outputs with q = k, o_t = S_t^T k_t = e^g S_{t-1}^T k_t + |k|^2 u_t
    kk = (k * k).sum(-1, keepdims=True)
    kk = np.repeat(kk, v.shape[2] // k.shape[2], 2)
    o = ref.gdr_fwd(k, k, v, g, b, S0)[0]
    bb = b[..., None]
    # o = w + kk u with u = b (v - w): w = (o - kk b v) / (1 - kk b) unless kk b = 1, where o = v and u <= |v| + |w|
    w = np.where(np.abs(1 - kk * bb) > 1e-3, (o - kk * bb * v) / np.where(np.abs(1 - kk * bb) > 1e-3, 1 - kk * bb, 1.0), o)
    u = bb * (np.abs(v) + np.abs(w))
    total = lambda x: np.sqrt((x * x).sum((1, 3)))
    y = r[2]
    un, yn, dn = (np.sqrt((x * x).sum(-1)) for x in (u, y, do))
    Sn = total(u) + (0 if S0 is None else np.sqrt((S0 * S0).sum((2, 3))))
    side = lambda a, s: np.sqrt((a * a).sum(1)) * s
    return side(dn, Sn), side(un, total(do) + total(y)) + side(yn, Sn)


def _check_grads(out, ins, dtype, T, S0, dS, cancels=False, reach=1):
    q, k, v, g, b, do = (_np(x) for x in ins)
    terms = []
    r = ref.gdr_bwd(q, k, v, g, b, do, S0, dS, terms)
    bf, fp = dtype == "bf16", _fp32(T, reach)
    scale = np.sqrt(T) * 0.1
    wide = _terms(q, k, v, g, b, do, S0, r) if cancels else (0.0, 0.0)
    _rel(out[0], r[0], 2.0 ** -6 if bf else fp, "dq", scale + wide[0])
    _rel(out[1], r[1], 2.0 ** -6 if bf else 2 * fp, "dk", scale + wide[1])
    _rel(out[2], r[2], 2.0 ** -7 if bf else fp, "dv", scale)
    if bf:
        _elem(out[2], r[2], fp, "dv")
    db = _np(out[4])
    tol = 2 * fp * (terms[0] + np.sqrt((terms[0] ** 2).mean(1, keepdims=True))) + 1e-30
    if bf:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -6) * (np.abs(r[4]) + terms[0])
    assert (np.abs(db - r[4]) <= tol).all(), ("d_beta", (np.abs(db - r[4]) / tol).max())
    _rel(out[5], r[5], fp, "d_initial_state", 1.0, (2, 3))
    # what the decay gradient's differences are taken of
    o = ref.gdr_fwd(q, k, v, g, b, S0)[0]
    w = np.sqrt(((do * o).sum(-1) ** 2 + (r[2] * v).sum(-1) ** 2).sum(1))
    dg = _np(out[3])
    err, ok = _norm(dg - r[3], 1), fp * (_norm(r[3], 1) + w) + 1e-30
    assert np.isfinite(dg).all() and (err <= ok).all(), ("d_log_decay", (err / ok).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 16, 63, 64, 65, 200])
def test_forward(T, dk, dv, dtype):
    _check_fwd(2, T, 2, 4, dk, dv, dtype, s0=T != 64, seed=T, beta=1.0 + T % 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 17, 64, 65, 200])
def test_backward(T, dk, dv, dtype):
    _check_bwd(2, T, 2, 4, dk, dv, dtype, s0=T != 64, seed=T, beta=1.0 + T % 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 129, 1, 1), (1, 777, 1, 3), (2, 511, 2, 4), (3, 1025, 5, 5), (1, 64 * 33 + 1, 1, 2)])
def test_longer_sequences_and_head_counts(B, T, Hk, H, dtype):
    _check_fwd(B, T, Hk, H, 128 if H < 4 else 64, 64, dtype, seed=T)
    _check_bwd(B, T, Hk, H, 64, 128 if H < 4 else 64, dtype, seed=T)


def test_eight_heads_of_one_key_head():
    _check_fwd(1, 150, 1, 8, 64, 64, "bf16", seed=3)
    _check_bwd(1, 150, 1, 8, 64, 64, "f32", seed=3)


def _edge(kind, B, T, H, dk, dv, dtype, Hk=None):
    import torch
    q, k, v, g, b, do = _inputs(B, T, Hk or H, H, dk, dv, dtype, seed=11, beta=2.0)
    u = torch.rand(B, T, H, generator=torch.Generator().manual_seed(5))
    inf = float("inf")
    if kind == "no decay":
        g = torch.zeros_like(g)
    if kind == "resets":
        g = torch.where(u < 0.05, torch.tensor(-inf), -0.02 * u)
    if kind == "cliffs":  # far below anything fp32 holds, next to slow decays
        g = torch.where(u < 0.03, torch.tensor(-1e30), torch.where(u < 0.1, -100.0 * u, -0.001 * u))
    if kind == "all reset":
        g = torch.full_like(g, -inf)
    if kind == "beta 0":
        b = torch.zeros_like(b)
    if kind == "some beta 0":
        b = torch.where(u < 0.5, torch.zeros_like(b), b)
    if kind in ("one key", "one key, reflected"):  # powers of the score matrix grow like binomials, its inverse does not
        k = k[:, :1].expand_as(k).contiguous()
        g = -0.001 * u
        b = torch.full_like(b, 1.0 if kind == "one key" else 2.0)
    if kind == "zero keys":
        k = torch.zeros_like(k)
    if kind == "large values":
        v = v * 2.0 ** 60
    if kind == "small values":
        v = v * 2.0 ** -60
    return q, k, v, g, b, do


KINDS = ["no decay", "resets", "cliffs", "all reset", "beta 0", "some beta 0", "one key", "one key, reflected", "zero keys"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_edges_forward(kind, dtype):
    _check_fwd(1, 200, 2, 2, 64, 64, dtype, ins=_edge(kind, 1, 200, 2, 64, 64, dtype), reach=64 if "reflected" in kind else 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_edges_backward(kind, dtype):
    out = _check_bwd(1, 200, 2, 2, 64, 64, dtype, ins=_edge(kind, 1, 200, 2, 64, 64, dtype), cancels="one key" in kind,
                     reach=64 if "reflected" in kind else 1)
    if kind == "all reset":
        assert float(out[3].abs().max()) == 0.0 and float(out[5].abs().max()) == 0.0


@pytest.mark.parametrize("kind", ["large values", "small values"])
def test_sizes_of_values(kind):
    """The rule is linear in v and the start state: scaled values give scaled outputs, bit for bit (powers of two)."""
    import torch
    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, _ = _edge("", 1, 150, 2, 64, 64, "bf16")
    f = 2.0 ** (60 if kind == "large values" else -60)
    o, s = kda.gdr_chunk_fwd(*_dev(q, k, v, g, b))
    o2, s2 = kda.gdr_chunk_fwd(*_dev(q, k, v * f, g, b))
    assert torch.equal(o2.float(), o.float() * f)
    # states keep terms of 2^-16 of them, which may pass under fp32's least at the small end
    assert torch.equal(s2, s * f)


def _cu(T):
    return [0, 0, 1, 64, 130, 130, 130 + 193, T - 70, T - 70]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_forward(dtype):
    """Sequences of no, one and many tokens back to back; rows behind the last stay as they were."""
    import torch
    import gated_delta_rule_78_amd as kda
    T, Hk, H, dk, dv = 700, 2, 4, 64, 128
    q, k, v, g, b, _ = _inputs(1, T, Hk, H, dk, dv, dtype, seed=9)
    cu = _cu(T)
    S0 = torch.randn(len(cu) - 1, H, dk, dv, generator=torch.Generator().manual_seed(1))
    mark = torch.full((1, T, H, dv), 7.0, dtype=q.dtype, device="cuda")
    o, sT = kda.gdr_chunk_fwd(*_dev(q, k, v, g, b), initial_state=S0.cuda(), out=mark,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert bool((o[0, cu[-1]:] == 7).all())
    parts = ref.packed(cu, ref.gdr_fwd, [_np(x) for x in (q, k, v, g, b)], [_np(S0)])
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if hi > lo:
            _out(o[:, lo:hi], parts[i][0], parts[i][1], dtype, hi - lo, i)
            _rel(sT[i:i + 1], parts[i][1], _fp32(hi - lo), i, 1.0, (2, 3))
        else:
            assert np.array_equal(_np(sT[i]), _np(S0[i]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_backward(dtype):
    import torch
    import gated_delta_rule_78_amd as kda
    T, Hk, H, dk, dv = 700, 2, 4, 128, 64
    ins = _inputs(1, T, Hk, H, dk, dv, dtype, seed=9)
    cu = _cu(T)
    gen = torch.Generator().manual_seed(1)
    S0, dS = (torch.randn(len(cu) - 1, H, dk, dv, generator=gen) for _ in range(2))
    out = kda.gdr_chunk_bwd(*_dev(*ins), initial_state=S0.cuda(), d_final_state=dS.cuda(),
                            cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    for x in out[:5]:
        assert bool((x[0, cu[-1]:] == 0).all())
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if lo == hi:
            assert np.array_equal(_np(out[5][i]), _np(dS[i]))
            continue
        part = [x[:, lo:hi] for x in ins]
        s, d = S0[i:i + 1], dS[i:i + 1]
        _check_grads([x[:, lo:hi] for x in out[:5]] + [out[5][i:i + 1]], part, dtype, hi - lo, _np(s), _np(d))


def test_packed_offsets_are_clamped():
    """Offsets out of range or out of order reach no memory but the batch's own."""
    import torch
    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, do = _dev(*_inputs(1, 300, 2, 2, 64, 64, "bf16"))
    good = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    bad = torch.tensor([-5, 100, 50, 1 << 30], dtype=torch.int32, device="cuda")
    for x, y in zip(kda.gdr_chunk_fwd(q, k, v, g, b, cu_seqlens=good), kda.gdr_chunk_fwd(q, k, v, g, b, cu_seqlens=bad)):
        assert torch.equal(x, y)
    for x, y in zip(kda.gdr_chunk_bwd(q, k, v, g, b, do, cu_seqlens=good), kda.gdr_chunk_bwd(q, k, v, g, b, do, cu_seqlens=bad)):
        assert torch.equal(x, y)


def test_no_tokens():
    import torch
    import gated_delta_rule_78_amd as kda
    z = lambda *s: torch.zeros(*s, device="cuda")
    s0 = torch.randn(2, 3, 64, 64, device="cuda")
    ins = (z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3), z(2, 0, 3))
    o, sT = kda.gdr_chunk_fwd(*ins, initial_state=s0)
    assert o.numel() == 0 and torch.equal(sT, s0)
    assert float(kda.gdr_chunk_fwd(*ins)[1].abs().max()) == 0.0
    assert torch.equal(kda.gdr_chunk_bwd(*ins, z(2, 0, 3, 64), d_final_state=s0)[5], s0)
    empty = (z(0, 5, 3, 64), z(0, 5, 3, 64), z(0, 5, 3, 64), z(0, 5, 3), z(0, 5, 3))
    assert kda.gdr_chunk_fwd(*empty)[1].shape == (0, 3, 64, 64)
    assert kda.gdr_chunk_bwd(*empty, empty[2])[5].shape == (0, 3, 64, 64)


def test_what_is_not_wanted():
    import torch
    import gated_delta_rule_78_amd as kda
    ins = _dev(*_inputs(1, 200, 2, 2, 64, 64, "bf16"))
    full = kda.gdr_chunk_bwd(*ins)
    some = kda.gdr_chunk_bwd(*ins, want_d_decay=False, want_d_initial=False)
    assert some[3] is None and some[5] is None
    for i in (0, 1, 2, 4):
        assert torch.equal(full[i], some[i])
    o, s = kda.gdr_chunk_fwd(*ins[:5], want_final=False)
    assert s is None and torch.equal(o, kda.gdr_chunk_fwd(*ins[:5])[0])


def test_prepared_queries_and_keys():
    import torch
    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, _ = _dev(*_inputs(1, 100, 2, 4, 64, 64, "bf16"))
    q, k = 3 * q, 2 * k
    qn, kn = kda.qk_norm_rope(q, k, norm="l2")
    for x, y in zip(kda.gdr_chunk_fwd(q, k, v, g, b, qk_prep=dict(norm="l2")), kda.gdr_chunk_fwd(qn, kn, v, g, b)):
        assert torch.equal(x, y)
    s = [torch.zeros(1, 4, 64, 64, device="cuda") for _ in range(3)]
    o = kda.gdr_decode_tokens(q, k, v, g, b, s[0], qk_prep=dict(norm="l2"))
    assert torch.equal(o, kda.gdr_decode_tokens(qn, kn, v, g, b, s[1])) and torch.equal(s[0], s[1])
    one = [x[:, 0].contiguous() for x in (q, k, v, g, b)]
    kda.gdr_decode_step(*one, s[2], qk_prep=dict(norm="l2"))


@pytest.mark.parametrize("T,packed", [(4096, False), (9000, True)])
def test_state_in_place_over_segments(T, packed):
    """final_state may be initial_state: a segment that ends early must not be read as the start."""
    import torch
    import gated_delta_rule_78_amd as kda
    H = 2
    q, k, v, g, b, _ = _dev(*_inputs(1, T, H, H, 64, 128, "bf16"))
    cu, n = None, 1
    if packed:
        cu = torch.tensor([0, 0, 64 * 120 + 1, 64 * 120 + 20, T], dtype=torch.int32, device="cuda")
        n = 4
    s0 = torch.randn(n, H, 64, 128, device="cuda")
    o, st = kda.gdr_chunk_fwd(q, k, v, g, b, initial_state=s0, cu_seqlens=cu)
    for _ in range(3):
        s = s0.clone()
        o2, st2 = kda.gdr_chunk_fwd(q, k, v, g, b, initial_state=s, final_state=s, cu_seqlens=cu)
        assert st2 is s and torch.equal(o, o2) and torch.equal(st, s)


@pytest.mark.parametrize("per", [1, 2, 3])
def test_forced_segments(per):
    """Every segment length in a process of its own (the variable is read once)."""
    code = (f"import sys; sys.path[:0] = [{HERE!r}, {ROOT!r}]\n"
            "from test_gpu_gdr import _check_fwd, _check_bwd, test_packed_forward as pf, test_packed_backward as pb, _edge\n"
            "for dt in ('bf16', 'f32'):\n"
            "    _check_fwd(2, 64 * 7 + 5, 1, 2, 128, 128, dt, beta=2.0); _check_fwd(1, 64 * 6, 2, 2, 64, 128, dt, s0=False)\n"
            "    _check_bwd(2, 64 * 7 + 5, 1, 2, 128, 64, dt, beta=2.0); _check_bwd(1, 64 * 5 + 1, 2, 2, 64, 128, dt, s0=False)\n"
            "    _check_fwd(1, 200, 2, 2, 64, 64, dt, ins=_edge('resets', 1, 200, 2, 64, 64, dt))\n"
            "    _check_bwd(1, 200, 2, 2, 64, 64, dt, ins=_edge('no decay', 1, 200, 2, 64, 64, dt))\n"
            "    pf(dt); pb(dt)\n"
            "    print('done', dt, flush=True)\n")
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, KDA_GDR_SEGMENT=str(per)), capture_output=True,
                       text=True, timeout=110)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("keep", [1100])
def test_decay_gradient_over_groups(keep, dtype):
    """Beyond 1,024 tokens the decay gradient's sums go over several groups of chunks."""
    _check_bwd(1, keep, 2, 2, 64, 64, dtype, seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_do_not_depend_on_timing(dtype):
    import torch
    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, do = _dev(*_inputs(2, 1000, 2, 4, 128, 128, dtype))
    one = (*kda.gdr_chunk_fwd(q, k, v, g, b), *kda.gdr_chunk_bwd(q, k, v, g, b, do))
    for _ in range(3):
        for x, y in zip(one, (*kda.gdr_chunk_fwd(q, k, v, g, b), *kda.gdr_chunk_bwd(q, k, v, g, b, do))):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    import torch
    import gated_delta_rule_78_amd as kda
    sets = [_dev(*_inputs(1, 1500 + 64 * i, 2, 4, 64, 128, "bf16", seed=i)) for i in range(2)]
    want = [(*kda.gdr_chunk_fwd(*s[:5]), *kda.gdr_chunk_bwd(*s)) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = (*kda.gdr_chunk_fwd(*sets[i][:5]), *kda.gdr_chunk_bwd(*sets[i]))
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        for a, b in zip(w, x):
            assert torch.equal(a, b)


@pytest.mark.parametrize("packed", [False, True])
def test_captured_and_replayed(packed):
    """Forward and backward in a captured graph, replayed on new inputs with eager work between."""
    import torch
    import gated_delta_rule_78_amd as kda
    T = 500
    ins = _dev(*_inputs(1, T, 2, 4, 64, 64, "bf16", seed=0))
    cu = torch.tensor([0, 3, 200, T], dtype=torch.int32, device="cuda") if packed else None
    call = lambda x: (*kda.gdr_chunk_fwd(*x[:5], cu_seqlens=cu), *kda.gdr_chunk_bwd(*x, cu_seqlens=cu))
    call(ins)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ins)
    for seed in (1, 2, 3):
        new = _dev(*_inputs(1, T, 2, 4, 64, 64, "bf16", seed=seed))
        want = call(new)
        for a, b in zip(ins, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bwd", [False, True])
def test_workspace_of_the_caller(bwd):
    """One's own workspace, whatever was in it, and no byte behind it."""
    import torch
    import gated_delta_rule_78_amd as kda
    ins = _dev(*_inputs(1, 2000, 1, 2, 64, 64, "bf16"))
    call = (lambda **k: kda.gdr_chunk_bwd(*ins, **k)) if bwd else (lambda **k: kda.gdr_chunk_fwd(*ins[:5], **k))
    want = call()
    from gated_delta_rule_78_amd.gdr import _planned
    need = _planned(*ins[:5], -1, bwd)[-1]
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    for a, b in zip(want, call(workspace=ws[:need])):
        assert torch.equal(a, b)
    assert bool((ws[need:] == 0xFF).all())
    with pytest.raises(kda.KdaError):
        call(workspace=ws[:need - 256])


def _steps(ins, S, upto=None):
    """(o, S) of the recurrence, fp64."""
    q, k, v, g, b = (_np(x) for x in ins)
    o, s = np.zeros(v.shape), _np(S)
    for i in range(v.shape[0]):
        n = v.shape[1] if upto is None else int(min(max(upto[i], 0), v.shape[1]))
        if n:
            x, y = ref.gdr_fwd(*(z[i:i + 1, :n] for z in (q, k, v, g, b)), s[i:i + 1])
            o[i:i + 1, :n], s[i:i + 1] = x, y
    return o, s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (3, 5, 2, 4), (2, 19, 3, 3), (129, 1, 16, 32)])
def test_decode(B, T, Hk, H, dk, dv, dtype):
    import torch
    import gated_delta_rule_78_amd as kda
    ins = _inputs(B, T, Hk, H, dk, dv, dtype, seed=T, beta=2.0)[:5]
    S = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(4))
    r, rs = _steps(ins, S)
    s = S.cuda()
    if T == 1:
        o = kda.gdr_decode_step(*(x[:, 0] for x in _dev(*ins)), s)[:, None]
    else:
        o = kda.gdr_decode_tokens(*_dev(*ins), s)
    tol = _fp32(64 * T)
    _rel(s, rs, tol, "state", 0.0, (2, 3))
    x = _np(o)
    assert (np.abs(x - r) <= (2.0 ** -8 * np.abs(r) if dtype == "bf16" else 0) + tol * 8 * np.abs(r).max()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_of_some_tokens(dtype):
    """counts, update=False and no queries; T over the eight tokens that are staged at a time."""
    import torch
    import gated_delta_rule_78_amd as kda
    B, T, Hk, H, dk, dv = 6, 11, 2, 4, 64, 128
    ins = _inputs(B, T, Hk, H, dk, dv, dtype, seed=8)[:5]
    S = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(4))
    counts = [0, 1, 8, 9, 11, 40]
    x, c = _dev(*ins), torch.tensor(counts, dtype=torch.int32, device="cuda")
    whole = S.cuda()
    o = kda.gdr_decode_tokens(*x, whole)
    s = S.cuda()
    assert torch.equal(kda.gdr_decode_tokens(*x, s, update=False), o) and torch.equal(s, S.cuda())
    mark = torch.full_like(o, 7.0)
    part = kda.gdr_decode_tokens(*x, s, counts=c, out=mark)
    alone = S.cuda()
    assert kda.gdr_decode_tokens(None, *x[1:], alone, counts=c) is None
    assert torch.equal(alone, s)
    for i, n in enumerate(counts):
        n = min(n, T)
        assert torch.equal(part[i, :n], o[i, :n]) and bool((part[i, n:] == 7).all())
    _, rs = _steps(ins, S, counts)
    _rel(s, rs, _fp32(64 * T), "state", 0.0, (2, 3))
    assert torch.equal(s[0], S[0].cuda()) and torch.equal(s[4:], whole[4:])
    none = S.cuda()
    kda.gdr_decode_tokens(*x, none, counts=torch.tensor([-3] * B, dtype=torch.int32, device="cuda"), out=mark.fill_(7.0))
    assert torch.equal(none, S.cuda()) and bool((mark == 7).all())


def test_decode_ignores_tokens_that_do_not_count():
    """Padding behind the counted tokens may hold anything."""
    import torch
    import gated_delta_rule_78_amd as kda
    x = _dev(*_inputs(2, 4, 2, 2, 64, 64, "bf16", seed=8)[:5])
    S = torch.randn(2, 2, 64, 64, device="cuda")
    c = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    a, b = S.clone(), S.clone()
    o = kda.gdr_decode_tokens(*x, a, counts=c)
    for y in x:
        y[0, 2:], y[1, 3:] = float("nan"), float("inf")
    p = kda.gdr_decode_tokens(*x, b, counts=c)
    assert torch.equal(a, b) and torch.equal(o[0, :2], p[0, :2]) and torch.equal(o[1, :3], p[1, :3])


def test_prefill_then_decode():
    """A prompt in chunks and its tokens one by one from there agree with the whole."""
    import torch
    import gated_delta_rule_78_amd as kda
    ins = _inputs(2, 140, 2, 4, 128, 128, "f32", seed=6)[:5]
    x = _dev(*ins)
    o, s = kda.gdr_chunk_fwd(*(y[:, :130].contiguous() for y in x))
    tail = [kda.gdr_decode_step(*(y[:, t].contiguous() for y in x), s) for t in range(130, 140)]
    r, rs = ref.gdr_fwd(*(_np(y) for y in ins))
    _rel(torch.cat([o, torch.stack(tail, 1)], 1), r, _fp32(140), "o", 1.0)
    _rel(s, rs, _fp32(140), "state", 1.0, (2, 3))


def test_other_sequences_keep_their_results():
    """A token that is not finite spoils its own sequence and head, from its chunk on, and nothing else."""
    import torch
    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, _ = _dev(*_inputs(2, 300, 2, 2, 64, 64, "bf16"))
    o, s = kda.gdr_chunk_fwd(q, k, v, g, b)
    v[0, 150, 0] = float("nan")
    o2, s2 = kda.gdr_chunk_fwd(q, k, v, g, b)
    assert torch.equal(o[1], o2[1]) and torch.equal(o[0, :, 1], o2[0, :, 1]) and torch.equal(o[0, :128, 0], o2[0, :128, 0])
    assert torch.equal(s[1], s2[1]) and torch.equal(s[0, 1], s2[0, 1])
    assert bool(torch.isnan(o2[0, 150:, 0]).all()) and bool(torch.isnan(s2[0, 0]).all())


@pytest.mark.parametrize("H,dk,dv,T,dtype,most", [(1, 128, 64, 131072, "bf16", 64), (1, 128, 128, 131072, "bf16", 64),
                                                  (2, 64, 64, 32768, "bf16", 64), (1, 128, 128, 9000, "f32", 24),
                                                  (1, 64, 128, 1200, "bf16", 3), (1, 64, 128, 700, "bf16", 1),
                                                  (1, 128, 64, 1000, "f32", 1)])  # 2 (8 + 0.5) steps against 16
def test_few_packed_chains_have_few_links(H, dk, dv, T, dtype, most):
    """Segments of one long packed sequence are joined one after another, so that there are about as many as a segment has
    chunks, at most 2.5 times the root of all; and a short one is walked whole.  The offsets kernel leaves 0, T
    and a segment's chunks at the end of the workspace.  The results are those of the sequence unpacked."""
    import torch
    import gated_delta_rule_78_amd as kda
    from gated_delta_rule_78_amd.gdr import _planned
    g = torch.Generator(device="cuda").manual_seed(7)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    unit = lambda *s: torch.nn.functional.normalize(rn(*s), dim=-1).to(dt)
    q, k, v, b = unit(1, T, H, dk), unit(1, T, H, dk), rn(1, T, H, dv).to(dt), torch.sigmoid(rn(1, T, H)).to(dt)
    gl = -0.1 * torch.rand(1, T, H, generator=g, device="cuda")
    s0 = rn(1, H, dk, dv)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ws = torch.zeros(_planned(q, k, v, gl, b, 1)[-1], dtype=torch.uint8, device="cuda")
    o, s = kda.gdr_chunk_fwd(q, k, v, gl, b, initial_state=s0, cu_seqlens=cu, workspace=ws)
    tail = ws[-65536:].view(torch.int32).tolist() if ws.numel() >= 65536 else ws.view(torch.int32).tolist()
    at = [i for i in range(len(tail) - 2) if tail[i] == 0 and tail[i + 1] == T]
    chunks = -(-T // 64)
    segments = {-(-chunks // tail[i + 2]) for i in at if tail[i + 2] > 0}
    assert segments and max(segments) <= min(most, max(1, 2.5 * chunks ** 0.5)), segments
    r, rs = kda.gdr_chunk_fwd(q, k, v, gl, b, initial_state=s0)
    _rel(s, _np(rs), 2 * _fp32(T), "final state", 1.0, (2, 3))
    if dtype == "bf16":  # two roundings of values that differ by fp32's bound: a step at most
        x, y = _np(o), _np(r)
        assert (np.abs(x - y) <= 2.0 ** -7 * np.abs(y) + 2 * (3 * 2.0 ** -16 + _fp32(T)) * 8).all()
    else:
        _rel(o, _np(r), 2 * _fp32(T), "o", 0.1 * np.sqrt(T))


def _rounded_dq_dk(q, k, v, g, b, do, S0, dS, scores=lambda x: x):
    """dq and dk in fp64 with a rounding to bf16 where the kernels have one: the state S that a chunk meets, the gradient R
    of the state behind it, r = v - e^g S^T k, y = dv, and the results.  scores: what a score is taken as."""
    import torch
    bf = lambda x: torch.from_numpy(np.ascontiguousarray(x)).float().bfloat16().double().numpy()
    B, T, Hk, dk = q.shape
    H, dv, C = *v.shape[2:], 64
    dq, dkk = np.zeros((B, T, H, dk)), np.zeros((B, T, H, dk))
    ys = ref.gdr_bwd(q, k, v, g, b, do, S0, dS)[2]
    for i, h in np.ndindex(B, H):
        Q, K, V, G, be, D, Y = (x[i, :, j] for x, j in ((q, h * Hk // H), (k, h * Hk // H), (v, h), (g, h), (b, h), (do, h), (ys, h)))
        S, R = (np.zeros((dk, dv)) if x is None else x[i, h] for x in (S0, dS))
        starts, behind, r = {}, {}, np.zeros((T, dv))
        for t in range(T):
            if t % C == 0:
                starts[t // C] = bf(S)
            S = np.exp(G[t]) * S
            r[t] = V[t] - S.T @ K[t]
            S = S + np.outer(K[t], be[t] * r[t])
        for t in range(T - 1, -1, -1):
            if t == T - 1 or (t + 1) % C == 0:
                behind[t // C] = bf(R)
            R = (np.exp(G[t + 1]) if t + 1 < T else 1.0) * R + np.outer(Q[t], D[t]) - np.outer(K[t], Y[t])
        for c in starts:
            s = slice(c * C, min(T, c * C + C))
            sums = np.cumsum(G[s])
            end = sums[-1] + (G[s.stop] if s.stop < T else 0.0)  # with the next token's decay
            low = np.tril(np.exp(np.minimum(sums[:, None] - sums, 0.0)))
            u, y, eg = be[s, None] * bf(r[s]), bf(Y[s]), np.exp(sums)[:, None]
            E, F = scores(low * (D[s] @ u.T)), scores(np.tril(low * (y @ u.T), -1))
            dq[i, s, h] = E @ K[s] + eg * (D[s] @ starts[c].T)
            dkk[i, s, h] = E.T @ Q[s] - (F + F.T) @ K[s] - eg * (y @ starts[c].T) + np.exp(end - sums)[:, None] * (u @ behind[c].T)
    share = lambda x: bf(x.reshape(B, T, Hk, H // Hk, dk).sum(3))
    return share(dq), share(dkk)


# B, T, Hk, H, dk, dv, start states and gradients of the last ones, largest beta
ROUNDED = [(1, 400, 2, 2, 128, 128, True, 1.0), (1, 400, 2, 4, 64, 64, True, 2.0), (1, 300, 4, 4, 64, 128, False, 1.0),
           (2, 200, 2, 4, 128, 64, True, 1.0)]


def _rounded_case(B, T, Hk, H, dk, dv, states, beta):
    import torch
    ins = _inputs(B, T, Hk, H, dk, dv, "bf16", T + dv, beta)
    gen = torch.Generator().manual_seed(dk)
    S0, dS = (torch.randn(B, H, dk, dv, generator=gen) for _ in range(2)) if states else (None, None)
    return ins, S0, dS


@pytest.mark.parametrize("B,T,Hk,H,dk,dv,states,beta", ROUNDED)
def test_gradients_of_q_and_k_take_no_other_roundings(B, T, Hk, H, dk, dv, states, beta):
    """bf16 inputs: dq and dk as fp64 gives them with the roundings that are named, and their distance from the formula's.

    From it: each of a sum's products has roundings of its own in one operand (dq: d_o S^T in S, E K in r) or two (dk:
    y S^T, F in y and r, u R^T), independent ones of at most 2^-8 / sqrt(3) in the root mean square, and the result has
    one: sqrt(2) 2^-8 / sqrt(3) and 2^-8 of the norm.  To the rounded form: an operand that is off by a share d before it
    is rounded to bf16 falls on the other side in d / step of all cases and is then a step off, sqrt(d step) in the
    root mean square with a step of up to 2^-7.  d is fp32's bound (_fp32, up to 8e-6 here) for the four operands, and 2^-16 of
    the scores for the result: (4 . 8e-6 2^-7 + 2^-16 2^-7)^(1/2) = 6.1e-4, within 2^-10."""
    import gated_delta_rule_78_amd as kda
    ins, S0, dS = _rounded_case(B, T, Hk, H, dk, dv, states, beta)
    out = kda.gdr_chunk_bwd(*_dev(*ins), initial_state=_dev(S0)[0], d_final_state=_dev(dS)[0])
    x = [_np(y) for y in ins]
    want, near = ref.gdr_bwd(*x, _np(S0), _np(dS)), _rounded_dq_dk(*x, _np(S0), _np(dS))
    for i, (name, bound) in enumerate((("dq", 2.0 ** -8 * np.sqrt(2 / 3)), ("dk", 2.0 ** -8))):
        _rel(out[i], want[i], bound, name)
        _rel(out[i], near[i], 2.0 ** -10, name + " as rounded")


def test_rounded_gradients_tell_scores_of_fewer_bits():
    """The bound to the rounded form is one that scores of 8 bits do not keep."""
    import torch
    bf = lambda x: torch.from_numpy(np.ascontiguousarray(x)).float().bfloat16().double().numpy()
    for case in ROUNDED:
        ins, S0, dS = _rounded_case(*case)
        x = [_np(y) for y in ins]
        good, bad = _rounded_dq_dk(*x, _np(S0), _np(dS)), _rounded_dq_dk(*x, _np(S0), _np(dS), bf)
        assert all((_norm(b - a, (1, 3)) / _norm(a, (1, 3))).max() > 2.0 ** -10 for a, b in zip(good, bad)), case


def test_decode_of_prepared_queries_and_keys():
    import torch
    import gated_delta_rule_78_amd as kda
    q, k, v, g, b, _ = (x[:, 0].contiguous() for x in _dev(*_inputs(3, 2, 2, 4, 64, 128, "bf16")))
    q, k = 3 * q, 2 * k
    qn, kn = (x[:, 0].contiguous() for x in kda.qk_norm_rope(q[:, None].contiguous(), k[:, None].contiguous(), norm="l2"))
    S = torch.randn(3, 4, 64, 128, device="cuda")
    a, c = S.clone(), S.clone()
    o = kda.gdr_decode_step(q, k, v, g, b, a, qk_prep=dict(norm="l2"))
    assert torch.equal(o, kda.gdr_decode_step(qn, kn, v, g, b, c)) and torch.equal(a, c) and not torch.equal(a, S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [700, 9000])
def test_packed_workspace_may_hold_anything(T, dtype):
    """Slots that no chunk, segment or token of a packed batch needs are not read: NaN patterns in all of the workspace."""
    import torch
    import gated_delta_rule_78_amd as kda
    from gated_delta_rule_78_amd.gdr import _planned
    ins = _dev(*_inputs(1, T, 1, 2, 64, 64, dtype))
    cu = _cu(T)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for bwd in (False, True):
        call = (lambda **kw: kda.gdr_chunk_bwd(*ins, cu_seqlens=c, **kw)) if bwd else (
            lambda **kw: kda.gdr_chunk_fwd(*ins[:5], cu_seqlens=c, out=torch.zeros_like(ins[2]), **kw))
        need = _planned(*ins[:5], len(cu) - 1, bwd)[-1]
        zeros, ws = torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        for x, y in zip(call(workspace=zeros), call(workspace=ws[:need])):
            assert torch.equal(x, y)
        assert bool((ws[need:] == 0xFF).all())


def test_decode_captured_and_replayed():
    """A round of drafting in a captured graph: outputs with the state left alone, then the state over the counted tokens."""
    import torch
    import gated_delta_rule_78_amd as kda
    ins = _dev(*_inputs(3, 5, 2, 4, 64, 128, "bf16")[:5])
    S, c = torch.zeros(3, 4, 64, 128, device="cuda"), torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")

    def call(x, S, c):
        o = kda.gdr_decode_tokens(*x, S, update=False)
        kda.gdr_decode_tokens(None, *x[1:], S, counts=c)
        return o

    call(ins, S, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ins, S, c)
    S.zero_()
    T = torch.zeros_like(S)
    for seed in (1, 2, 3):
        new, n = _dev(*_inputs(3, 5, 2, 4, 64, 128, "bf16", seed)[:5]), torch.tensor([seed, 5, 0], dtype=torch.int32, device="cuda")
        want = call(new, T, n)
        for a, b in zip((*ins, c), (*new, n)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(S, T)


def test_packed_batch_of_no_tokens():
    """Sequences without a token hand their states on, both ways."""
    import torch
    import gated_delta_rule_78_amd as kda
    z = lambda *s: torch.zeros(*s, device="cuda")
    ins = (z(1, 0, 2, 64), z(1, 0, 2, 64), z(1, 0, 4, 128), z(1, 0, 4), z(1, 0, 4))
    s = torch.randn(3, 4, 64, 128, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert torch.equal(kda.gdr_chunk_fwd(*ins, initial_state=s, cu_seqlens=cu)[1], s)
    assert torch.equal(kda.gdr_chunk_bwd(*ins, ins[2], d_final_state=s, cu_seqlens=cu)[5], s)
    assert kda.gdr_chunk_fwd(*ins, cu_seqlens=cu[:1])[1].shape == (0, 4, 64, 128)

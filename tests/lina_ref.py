"""Plain fp64 references of linear attention with a decay per head (token after token) and of
the query / key norm and rotation, and the error bounds their tests use."""
from __future__ import annotations

import numpy as np


def expand(x, H):
    """[.., Hk, d] -> [.., H, d]: head h goes with shared head h // (H // Hk)."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def lina_fwd(q, k, v, g, s0=None):
    """One batch: q, k [B,T,Hk,dk], v [B,T,H,dv], g [B,T,H] -> o, S_T, all fp64."""
    B, T, H, dv = v.shape
    q, k = expand(q, H).astype(np.float64), expand(k, H).astype(np.float64)
    v = v.astype(np.float64)
    S = np.zeros((B, H, q.shape[-1], dv)) if s0 is None else s0.astype(np.float64).copy()
    o = np.zeros((B, T, H, dv))
    for t in range(T):
        with np.errstate(invalid="ignore"):
            S = np.exp(g[:, t].astype(np.float64))[..., None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = np.einsum("bhij,bhi->bhj", S, q[:, t])
    return o, S


def lina_bwd(q, k, v, g, d_o, s0=None, d_sT=None):
    """Gradients token after token, from the recurrence's own derivative:
    R_t = dL/dS_t = q_t do_t^T + e^(g_(t+1)) R_(t+1)."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[-2:]
    qe, ke = expand(q, H).astype(np.float64), expand(k, H).astype(np.float64)
    v, u = v.astype(np.float64), d_o.astype(np.float64)
    a = np.exp(g.astype(np.float64))
    S = np.zeros((T + 1, B, H, dk, dv))
    if s0 is not None:
        S[0] = s0
    for t in range(T):
        S[t + 1] = a[:, t, :, None, None] * S[t] + ke[:, t, :, :, None] * v[:, t, :, None, :]
    R = np.zeros((B, H, dk, dv)) if d_sT is None else d_sT.astype(np.float64).copy()
    dq, dkk, dvv, dg = np.zeros_like(qe), np.zeros_like(ke), np.zeros_like(v), np.zeros((B, T, H))
    for t in range(T - 1, -1, -1):
        R = R + qe[:, t, :, :, None] * u[:, t, :, None, :]
        dq[:, t] = np.einsum("bhij,bhj->bhi", S[t + 1], u[:, t])
        dkk[:, t] = np.einsum("bhij,bhj->bhi", R, v[:, t])
        dvv[:, t] = np.einsum("bhij,bhi->bhj", R, ke[:, t])
        dg[:, t] = a[:, t] * (R * S[t]).sum((-1, -2))
        R = a[:, t, :, None, None] * R
    r = H // Hk
    share = lambda x: x.reshape(B, T, Hk, r, x.shape[-1]).sum(3)
    return share(dq), share(dkk), dvv, dg, R


def packed(cu, fn, *ins, states=()):
    """fn on every sequence of a packed batch; ins [1,T,...], states [N,...] (or None)."""
    outs = []
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        outs.append(fn(*[x[:, lo:hi] for x in ins], *[None if s is None else s[i:i + 1] for s in states]))
    return outs


def rotate(x, pos, inv, sections, interleaved, sign=1.0):
    """x [n, H, d], pos [axes, n]."""
    m = len(inv)
    if m == 0:
        return x
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = pos[axis].T.astype(np.float64) * inv[None]
    c, s = np.cos(ang)[:, None], sign * np.sin(ang)[:, None]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:2 * m:2], x[..., 1:2 * m:2]
        y[..., 0:2 * m:2], y[..., 1:2 * m:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :m], x[..., m:2 * m]
        y[..., :m], y[..., m:2 * m] = a * c - b * s, b * c + a * s
    return y


def rnorm(x, norm, eps):
    if norm is None:
        return np.ones(x.shape[:-1] + (1,))
    s = (x * x).sum(-1, keepdims=True)
    return 1.0 / np.sqrt((s / x.shape[-1] if norm == "rms" else s) + eps)


def qk_fwd(x, w, pos, inv, sections, interleaved, norm, eps):
    x = x.astype(np.float64)
    y = x * rnorm(x, norm, eps) * (1.0 if w is None else w.astype(np.float64))
    return rotate(y, pos, inv, sections, interleaved)


def qk_bwd(dy, x, w, pos, inv, sections, interleaved, norm, eps):
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    w = np.ones(x.shape[-1]) if w is None else w.astype(np.float64)
    z = rotate(dy, pos, inv, sections, interleaved, -1.0)
    r = rnorm(x, norm, eps)
    dw = (z * x * r).sum((0, 1))
    u = z * w
    if norm is None:
        return u, dw
    c = (x * u).sum(-1, keepdims=True) * r * r
    return r * (u - x * (c / x.shape[-1] if norm == "rms" else c)), dw

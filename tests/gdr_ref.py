"""Plain fp64 references of the gated delta rule with one decay per head (token after token) and of
drafted tokens' verification."""
from __future__ import annotations

import numpy as np

from lina_ref import expand


def gdr_fwd(q, k, v, g, b, s0=None):
    """q, k [B,T,Hk,dk], v [B,T,H,dv], g, b [B,T,H] -> o, S_T, all fp64."""
    B, T, H, dv = v.shape
    q, k = expand(q, H).astype(np.float64), expand(k, H).astype(np.float64)
    v, g, b = v.astype(np.float64), g.astype(np.float64), b.astype(np.float64)
    S = np.zeros((B, H, q.shape[-1], dv)) if s0 is None else s0.astype(np.float64).copy()
    o = np.zeros((B, T, H, dv))
    for t in range(T):
        S = np.exp(g[:, t])[..., None, None] * S
        u = b[:, t, :, None] * (v[:, t] - np.einsum("bhij,bhi->bhj", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        o[:, t] = np.einsum("bhij,bhi->bhj", S, q[:, t])
    return o, S


def gdr_bwd(q, k, v, g, b, d_o, s0=None, d_sT=None, terms=None):
    """Gradients token after token, from the recurrence's own derivative, in the order dq, dk, dv, dg, db, dS_0.
    terms: a list that gets db with every product's magnitude, sum |z_c r_c|."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[-2:]
    qe, ke = expand(q, H).astype(np.float64), expand(k, H).astype(np.float64)
    v, do, b = v.astype(np.float64), d_o.astype(np.float64), b.astype(np.float64)
    a = np.exp(g.astype(np.float64))
    S = np.zeros((T + 1, B, H, dk, dv))
    if s0 is not None:
        S[0] = s0
    for t in range(T):
        D = a[:, t, :, None, None] * S[t]
        u = b[:, t, :, None] * (v[:, t] - np.einsum("bhij,bhi->bhj", D, ke[:, t]))
        S[t + 1] = D + ke[:, t, :, :, None] * u[:, :, None, :]
    R = np.zeros((B, H, dk, dv)) if d_sT is None else d_sT.astype(np.float64).copy()
    size = np.zeros((B, T, H))
    dq, dkk, dvv, dg, db = np.zeros_like(qe), np.zeros_like(ke), np.zeros_like(v), np.zeros((B, T, H)), np.zeros((B, T, H))
    for t in range(T - 1, -1, -1):
        kt, D = ke[:, t], a[:, t, :, None, None] * S[t]
        R = R + qe[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = np.einsum("bhij,bhj->bhi", S[t + 1], do[:, t])
        r = v[:, t] - np.einsum("bhij,bhi->bhj", D, kt)
        z = np.einsum("bhij,bhi->bhj", R, kt)
        db[:, t], size[:, t] = (z * r).sum(-1), np.abs(z * r).sum(-1)
        y, u = b[:, t, :, None] * z, b[:, t, :, None] * r
        dvv[:, t] = y
        dkk[:, t] = np.einsum("bhij,bhj->bhi", R, u) - np.einsum("bhij,bhj->bhi", D, y)
        R = R - kt[..., :, None] * y[..., None, :]
        dg[:, t] = (R * D).sum((-1, -2))
        R = a[:, t, :, None, None] * R
    share = lambda x: x.reshape(B, T, Hk, H // Hk, x.shape[-1]).sum(3)
    if terms is not None:
        terms.append(size)
    return share(dq), share(dkk), dvv, dg, db, R


def packed(cu, fn, ins, states):
    """fn on every sequence of a packed batch; ins [1,T,...], states [N,...] (or None)."""
    return [fn(*[x[:, lo:hi] for x in ins], *[None if s is None else s[i:i + 1] for s in states])
            for i, (lo, hi) in enumerate(zip(cu, cu[1:]))]


def weights(x):
    x = np.asarray(x, dtype=np.float64)
    return np.where(np.isfinite(x) & (x > 0), x, 0.0)


def verify(p, drafts, q, u, u_next):
    """p [B,K+1,V], drafts [B,K], q [B,K,V] or None, u [B,K], u_next [B] -> accepted, next token."""
    B, K = drafts.shape
    V = p.shape[-1]
    ns, ts = [], []
    for i in range(B):
        n, w = 0, None
        while n < K and 0 <= drafts[i, n] < V:
            x = drafts[i, n]
            qx = 1.0 if q is None else float(q[i, n, x])
            if float(u[i, n]) * qx < float(p[i, n, x]):
                n += 1
                continue
            less = weights(q[i, n]) if q is not None else np.eye(1, V, x)[0]
            w = np.maximum(weights(p[i, n]) - less, 0.0)
            break
        if w is None or not w.sum() > 0:
            w = weights(p[i, n])
        c = np.cumsum(w)
        some = np.flatnonzero(w > 0)
        over = np.flatnonzero((c > float(u_next[i]) * c[-1]) & (w > 0))
        ns.append(n)
        ts.append(-1 if some.size == 0 else over[0] if over.size else some[-1])
    return np.array(ns), np.array(ts)

"""Gated delta rule with one decay per head: binding of the ``kda_gdr_*`` entry points.

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t

The rule of ``chunk_fwd`` with one gate for all key channels of a head, given as its logarithm, and
with q and k heads that serve several value heads if wanted; the states have the same layout.  Nothing is
normalised or scaled inside (see ``qk_norm_rope``: the rule asks for unit keys) and there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import functools

import gated_delta_rule_78_amd as _kda

from .lina import _sequences, _states, _workspace


@functools.lru_cache(maxsize=1024)
def _plan(q, k, v, log_decay, beta, n, bwd):
    """Checks shared by every form, once for the sizes they look at.  q (or None), k, v, log_decay, beta:
    (shape, dtype); n: sequences of a packed batch, or -1.  Returns (Hk, H, dk, dv, C shape, bytes of workspace)."""
    torch = _kda._torch()
    (ks, dtype), (vs, vt) = k, v
    lead = tuple(ks[:-2])
    if len(ks) not in (3, 4) or len(vs) != len(ks):
        raise ValueError("q, k, v are [B,T,heads,channels], or [B,heads,channels] for one token")
    Hk, dk = ks[-2:]
    H, dv = vs[-2:]
    code = _kda._dtype_code_of(dtype)
    for t, nm in ((q, "q"), (v, "v"), (beta, "beta")):
        if t is not None and t[1] != dtype:
            raise TypeError(f"{nm} must have the dtype of k")
    if (q is not None and q[0] != ks) or tuple(vs[:-2]) != lead or Hk < 1 or H % max(Hk, 1) != 0:
        raise ValueError("shapes: q, k [..., Hk, dk]; v [..., H, dv] with H a multiple of Hk")
    if log_decay[1] != torch.float32:
        raise TypeError("log_decay must be float32")
    if tuple(log_decay[0]) != (*lead, H) or tuple(beta[0]) != (*lead, H):
        raise ValueError("log_decay, beta: [..., H] as v")
    shape = _kda.Shape(lead[0], lead[1] if len(lead) > 1 else 1, H, dk, dv, 64, code)
    ref = ctypes.byref(shape)
    L = _kda.lib()
    kind = "bwd" if bwd else "fwd"
    if n < 0:
        need = getattr(L, f"kda_gdr_chunk_{kind}_workspace_size")(ref)
    else:
        need = getattr(L, f"kda_gdr_chunk_{kind}_varlen_workspace_size")(ref, n)
    return Hk, H, dk, dv, shape, int(need)


def _planned(q, k, v, log_decay, beta, n=-1, bwd=False):
    return _plan(None if q is None else (q.shape, q.dtype), (k.shape, k.dtype), (v.shape, v.dtype),
                 (log_decay.shape, log_decay.dtype), (beta.shape, beta.dtype), n, bwd)


def gdr_chunk_fwd(q, k, v, log_decay, beta, initial_state=None, out=None, final_state=None, want_final=True,
                  cu_seqlens=None, workspace=None, qk_prep=None):
    """Chunked forward over whole sequences.  q, k [B,T,Hk,dk], v [B,T,H,dv] and beta [B,T,H] (all bf16
    or all fp32, contiguous; Hk divides H, head h of v goes with head h // (H // Hk) of q and k); log_decay
    fp32 [B,T,H]; initial_state fp32 [B,H,dk,dv] or None.  cu_seqlens (int32 [N+1] on the device): a
    packed batch, B == 1, states [N,H,dk,dv]; tokens after the last offset are not written.  qk_prep:
    keyword arguments of qk_norm_rope, with which q and k are prepared first, or None.  Returns
    (o [B,T,H,dv], final_state fp32 or None)."""
    torch = _kda._torch()
    q, k = _kda._prepared(q, k, qk_prep)
    n = _sequences(q, cu_seqlens)
    Hk, H, dk, dv, shape, need = _planned(q, k, v, log_decay, beta, -1 if cu_seqlens is None else n)
    dev = q.device
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=dev)
    elif out.dtype != q.dtype or out.shape != v.shape:
        raise ValueError("out must be [B,T,H,dv] in the dtype of q")
    if final_state is None and want_final:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=dev)
    _states(((initial_state, "initial_state"), (final_state, "final_state")), n, H, dk, dv)
    workspace, nbytes = _workspace(need, workspace, dev)
    _kda._check((q, k, v, log_decay, beta, cu_seqlens, initial_state, out, final_state, workspace),
                ("q", "k", "v", "log_decay", "beta", "cu_seqlens", "initial_state", "out", "final_state", "workspace"),
                dev)
    p = _kda._addr
    args = (p(q), p(k), p(v), p(log_decay), p(beta), p(initial_state), p(out), p(final_state), p(workspace), nbytes)
    if cu_seqlens is None:
        _kda._launch("kda_gdr_chunk_fwd", dev, ctypes.byref(shape), Hk, *args)
    else:
        _kda._launch("kda_gdr_chunk_fwd_varlen", dev, ctypes.byref(shape), Hk, p(cu_seqlens), n, *args)
    return out, final_state


def gdr_chunk_bwd(q, k, v, log_decay, beta, d_o, initial_state=None, d_final_state=None, want_d_decay=True,
                  want_d_initial=True, cu_seqlens=None, workspace=None):
    """Gradients of L = sum <d_o, o> + <d_final_state, S_T> through gdr_chunk_fwd, which is recomputed
    inside.  Inputs as gdr_chunk_fwd; d_o [B,T,H,dv] in the dtype of q; d_final_state fp32
    [B or N,H,dk,dv] or None (zeros).  Returns (dq, dk, dv, d_log_decay or None, d_beta,
    d_initial_state or None): dq, dk, dv, d_beta in the shape and dtype of q, k, v, beta (shared heads
    get the sum), d_log_decay and d_initial_state fp32.  Tokens of a packed batch after the last
    offset get zeros."""
    torch = _kda._torch()
    n = _sequences(q, cu_seqlens)
    Hk, H, dk, dv, shape, need = _planned(q, k, v, log_decay, beta, -1 if cu_seqlens is None else n, True)
    if d_o.dtype != q.dtype or d_o.shape != v.shape:
        raise ValueError("d_o must be [B,T,H,dv] in the dtype of q")
    _states(((initial_state, "initial_state"), (d_final_state, "d_final_state")), n, H, dk, dv)
    dev = q.device
    new = torch.zeros_like if cu_seqlens is not None else torch.empty_like
    gq, gk, gv, gb = new(q), new(k), new(v), new(beta)
    gd = new(log_decay) if want_d_decay else None
    gs = torch.empty((n, H, dk, dv), dtype=torch.float32, device=dev) if want_d_initial else None
    workspace, nbytes = _workspace(need, workspace, dev)
    _kda._check((q, k, v, log_decay, beta, d_o, cu_seqlens, initial_state, d_final_state, workspace),
                ("q", "k", "v", "log_decay", "beta", "d_o", "cu_seqlens", "initial_state", "d_final_state",
                 "workspace"), dev)
    p = _kda._addr
    args = (p(q), p(k), p(v), p(log_decay), p(beta), p(initial_state), p(d_o), p(d_final_state), p(gq), p(gk), p(gv),
            p(gd), p(gb), p(gs), p(workspace), nbytes)
    if cu_seqlens is None:
        _kda._launch("kda_gdr_chunk_bwd", dev, ctypes.byref(shape), Hk, *args)
    else:
        _kda._launch("kda_gdr_chunk_bwd_varlen", dev, ctypes.byref(shape), Hk, p(cu_seqlens), n, *args)
    return gq, gk, gv, gd, gb, gs


def _decoded(q, k, v, log_decay, beta, state, out, dims):
    """Checks of a decode call: (Hk, C shape, out or None)."""
    torch = _kda._torch()
    if k.dim() != dims:
        raise ValueError(f"q, k, v have {dims} dimensions")
    Hk, H, dk, dv, shape, _ = _planned(q, k, v, log_decay, beta)
    _states(((state, "state"),), k.shape[0], H, dk, dv)
    if q is None:
        if out is not None:
            raise ValueError("out without q")
    elif out is None:
        out = torch.empty_like(v)
    elif out.dtype != v.dtype or out.shape != v.shape:
        raise ValueError("out must have the shape of v and the dtype of q")
    return Hk, shape, out


def gdr_decode_step(q, k, v, log_decay, beta, state, out=None, qk_prep=None):
    """One recurrent token for every (b, h): q, k [B,Hk,dk]; v [B,H,dv]; log_decay fp32 and beta
    [B,H]; state fp32 [B,H,dk,dv] updated in place; qk_prep as gdr_chunk_fwd.  Returns o [B,H,dv]."""
    q, k = _kda._prepared(q, k, qk_prep)
    Hk, shape, out = _decoded(q, k, v, log_decay, beta, state, out, 3)
    dev = k.device
    _kda._check((q, k, v, log_decay, beta, state, out), ("q", "k", "v", "log_decay", "beta", "state", "out"), dev)
    p = _kda._addr
    _kda._launch("kda_gdr_decode_step", dev, ctypes.byref(shape), Hk, p(q), p(k), p(v), p(log_decay), p(beta), p(state),
                 p(out))
    return out


def gdr_decode_tokens(q, k, v, log_decay, beta, state, out=None, counts=None, update=True, qk_prep=None):
    """Several tokens per (b, h) with the state read (and written) once: q, k [B,T,Hk,dk]; v [B,T,H,dv];
    log_decay fp32 and beta [B,T,H]; state fp32 [B,H,dk,dv].  counts (int32 [B] on the device, 0 to T;
    others count as the nearer end): of sequence b only the first counts[b] tokens are taken, the
    outputs behind them are left as they were.  update=False: the state stays as it is (outputs of
    drafted tokens, some of which may not stand).  q=None: no outputs, the state alone goes on (over the
    tokens that stand); qk_prep as gdr_chunk_fwd (needs q).  Returns o [B,T,H,dv], or None without q."""
    torch = _kda._torch()
    if qk_prep is not None:
        if q is None:
            raise ValueError("qk_prep without q: prepare k with qk_norm_rope first")
        q, k = _kda._prepared(q, k, qk_prep)
    if q is None and not update:
        raise ValueError("neither outputs (q) nor an update are asked for")
    Hk, shape, out = _decoded(q, k, v, log_decay, beta, state, out, 4)
    if counts is not None and (counts.dtype != torch.int32 or counts.shape != (k.shape[0],)):
        raise TypeError("counts must be an int32 tensor [B]")
    dev = k.device
    _kda._check((q, k, v, log_decay, beta, state, out, counts),
                ("q", "k", "v", "log_decay", "beta", "state", "out", "counts"), dev)
    p = _kda._addr
    _kda._launch("kda_gdr_decode_tokens", dev, ctypes.byref(shape), Hk, p(counts), 1 if update else 0, p(q), p(k), p(v),
                 p(log_decay), p(beta), p(state), p(out))
    return out

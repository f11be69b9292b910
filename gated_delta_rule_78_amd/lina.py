"""Linear attention with a decay per head: binding of the ``kda_lina_*`` entry points.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t

The delta rule of the other entry points without its erase term, with one gate per head; the
states have the same layout.  As everywhere here, nothing is normalised or scaled inside (see
``qk_norm_rope`` for q and k) and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools

import gated_delta_rule_78_amd as _kda


@functools.lru_cache(maxsize=1024)
def _plan(q, k, v, log_decay, n, bwd):
    """Checks shared by every form, once for the sizes they look at.  q, k, v, log_decay: (shape, dtype);
    n: sequences of a packed batch, or -1.  Returns (Hk, H, dk, dv, per_head, C shape, bytes of workspace)."""
    torch = _kda._torch()
    (qs, dtype), (vs, vt) = q, v
    lead = tuple(qs[:-2])
    if len(qs) not in (3, 4) or len(vs) != len(qs):
        raise ValueError("q, k, v are [B,T,heads,channels], or [B,heads,channels] for one token")
    Hk, dk = qs[-2:]
    H, dv = vs[-2:]
    code = _kda._dtype_code_of(dtype)
    for t, nm in ((k[1], "k"), (vt, "v")):
        if t != dtype:
            raise TypeError(f"{nm} must have the dtype of q")
    if k[0] != qs or tuple(vs[:-2]) != lead or Hk < 1 or H % max(Hk, 1) != 0:
        raise ValueError("shapes: q, k [..., Hk, dk]; v [..., H, dv] with H a multiple of Hk")
    if log_decay[1] != torch.float32:
        raise TypeError("log_decay must be float32")
    per_head = len(log_decay[0]) == 1
    if tuple(log_decay[0]) != ((H,) if per_head else (*lead, H)):
        raise ValueError("log_decay: [..., H] as v, or [H]")
    shape = _kda.Shape(lead[0], lead[1] if len(lead) > 1 else 1, H, dk, dv, 64, code)
    ref = ctypes.byref(shape)
    L = _kda.lib()
    if bwd:
        need = L.kda_lina_chunk_bwd_workspace_size(ref, Hk) if n < 0 else \
            L.kda_lina_chunk_bwd_varlen_workspace_size(ref, Hk, n)
    else:
        need = L.kda_lina_chunk_fwd_workspace_size(ref) if n < 0 else \
            L.kda_lina_chunk_fwd_varlen_workspace_size(ref, n)
    return Hk, H, dk, dv, per_head, shape, int(need)


def _planned(q, k, v, log_decay, n=-1, bwd=False):
    return _plan((q.shape, q.dtype), (k.shape, k.dtype), (v.shape, v.dtype), (log_decay.shape, log_decay.dtype), n, bwd)


def _states(ts, n, H, dk, dv):
    torch = _kda._torch()
    for t, nm in ts:
        if t is not None and (t.dtype != torch.float32 or t.shape != (n, H, dk, dv)):
            raise ValueError(f"{nm} must be float32 [{n},{H},{dk},{dv}]")


def _sequences(q, cu_seqlens):
    torch = _kda._torch()
    if q.dim() != 4:
        raise ValueError("q, k are [B,T,heads,channels]")
    if cu_seqlens is None:
        return q.shape[0]
    if q.shape[0] != 1:
        raise ValueError("a packed batch has B == 1")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor")
    return cu_seqlens.numel() - 1


def _workspace(need, workspace, dev):
    torch = _kda._torch()
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def lina_chunk_fwd(q, k, v, log_decay, initial_state=None, out=None, final_state=None, want_final=True,
                   cu_seqlens=None, workspace=None, qk_prep=None):
    """Chunked forward over whole sequences.  q, k [B,T,Hk,dk] and v [B,T,H,dv] (all bf16 or all
    fp32, contiguous; Hk divides H, head h of v goes with head h // (H // Hk) of q and k);
    log_decay fp32 [B,T,H], or [H] for a fixed decay per head; initial_state fp32 [B,H,dk,dv] or
    None.  cu_seqlens (int32 [N+1] on the device): a packed batch, B == 1, states [N,H,dk,dv];
    tokens after the last offset are not written.  qk_prep: keyword arguments of qk_norm_rope, with
    which q and k are prepared first, or None.  Returns (o [B,T,H,dv], final_state fp32 or
    None)."""
    torch = _kda._torch()
    q, k = _kda._prepared(q, k, qk_prep)
    n = _sequences(q, cu_seqlens)
    Hk, H, dk, dv, per_head, shape, need = _planned(q, k, v, log_decay, -1 if cu_seqlens is None else n)
    dev = q.device
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=dev)
    elif out.dtype != q.dtype or out.shape != v.shape:
        raise ValueError("out must be [B,T,H,dv] in the dtype of q")
    if final_state is None and want_final:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=dev)
    _states(((initial_state, "initial_state"), (final_state, "final_state")), n, H, dk, dv)
    workspace, nbytes = _workspace(need, workspace, dev)
    _kda._check((q, k, v, log_decay, cu_seqlens, initial_state, out, final_state, workspace),
                ("q", "k", "v", "log_decay", "cu_seqlens", "initial_state", "out", "final_state", "workspace"), dev)
    p = _kda._addr
    args = (p(q), p(k), p(v), p(log_decay), per_head, p(initial_state), p(out), p(final_state), p(workspace), nbytes)
    if cu_seqlens is None:
        _kda._launch("kda_lina_chunk_fwd", dev, ctypes.byref(shape), Hk, *args)
    else:
        _kda._launch("kda_lina_chunk_fwd_varlen", dev, ctypes.byref(shape), Hk, p(cu_seqlens), n, *args)
    return out, final_state


def lina_chunk_bwd(q, k, v, log_decay, d_o, initial_state=None, d_final_state=None, want_d_decay=True,
                   want_d_initial=True, cu_seqlens=None, workspace=None):
    """Gradients of L = sum <d_o, o> + <d_final_state, S_T> through lina_chunk_fwd, which is
    recomputed inside.  Inputs as lina_chunk_fwd; d_o [B,T,H,dv] in the dtype of q;
    d_final_state fp32 [B or N,H,dk,dv] or None (zeros).  Returns (dq, dk, dv, d_log_decay or
    None, d_initial_state or None): dq, dk, dv in the shape and dtype of q, k, v (shared heads
    get the sum), d_log_decay fp32 in the shape of log_decay, d_initial_state fp32.  Tokens of a
    packed batch after the last offset get zeros."""
    torch = _kda._torch()
    n = _sequences(q, cu_seqlens)
    Hk, H, dk, dv, per_head, shape, need = _planned(q, k, v, log_decay, -1 if cu_seqlens is None else n, True)
    if d_o.dtype != q.dtype or d_o.shape != v.shape:
        raise ValueError("d_o must be [B,T,H,dv] in the dtype of q")
    _states(((initial_state, "initial_state"), (d_final_state, "d_final_state")), n, H, dk, dv)
    dev = q.device
    new = torch.zeros_like if cu_seqlens is not None else torch.empty_like
    gq, gk, gv = new(q), new(k), new(v)
    gd = new(log_decay) if want_d_decay else None
    gs = torch.empty((n, H, dk, dv), dtype=torch.float32, device=dev) if want_d_initial else None
    workspace, nbytes = _workspace(need, workspace, dev)
    _kda._check((q, k, v, log_decay, d_o, cu_seqlens, initial_state, d_final_state, workspace),
                ("q", "k", "v", "log_decay", "d_o", "cu_seqlens", "initial_state", "d_final_state", "workspace"), dev)
    p = _kda._addr
    args = (p(q), p(k), p(v), p(log_decay), per_head, p(initial_state), p(d_o), p(d_final_state), p(gq), p(gk), p(gv),
            p(gd), p(gs), p(workspace), nbytes)
    if cu_seqlens is None:
        _kda._launch("kda_lina_chunk_bwd", dev, ctypes.byref(shape), Hk, *args)
    else:
        _kda._launch("kda_lina_chunk_bwd_varlen", dev, ctypes.byref(shape), Hk, p(cu_seqlens), n, *args)
    return gq, gk, gv, gd, gs


def _decode(entry, q, k, v, log_decay, state, out, dims):
    torch = _kda._torch()
    if q.dim() != dims:
        raise ValueError(f"q, k, v have {dims} dimensions")
    Hk, H, dk, dv, per_head, shape, _ = _planned(q, k, v, log_decay)
    _states(((state, "state"),), q.shape[0], H, dk, dv)
    dev = q.device
    if out is None:
        out = torch.empty_like(v)
    elif out.dtype != q.dtype or out.shape != v.shape:
        raise ValueError("out must have the shape of v and the dtype of q")
    _kda._check((q, k, v, log_decay, state, out), ("q", "k", "v", "log_decay", "state", "out"), dev)
    p = _kda._addr
    _kda._launch(entry, dev, ctypes.byref(shape), Hk, p(q), p(k), p(v), p(log_decay), per_head, p(state), p(out))
    return out


def lina_decode_step(q, k, v, log_decay, state, out=None, qk_prep=None):
    """One recurrent token for every (b, h): q, k [B,Hk,dk]; v [B,H,dv]; log_decay fp32 [B,H] or
    [H]; state fp32 [B,H,dk,dv] updated in place; qk_prep as lina_chunk_fwd.  Returns o [B,H,dv]."""
    q, k = _kda._prepared(q, k, qk_prep)
    return _decode("kda_lina_decode_step", q, k, v, log_decay, state, out, 3)


def lina_decode_tokens(q, k, v, log_decay, state, out=None, qk_prep=None):
    """Several tokens per (b, h) with the state read and written once: q, k [B,T,Hk,dk];
    v [B,T,H,dv]; log_decay fp32 [B,T,H] or [H]; state fp32 [B,H,dk,dv] in place.
    qk_prep as lina_chunk_fwd.  Returns o [B,T,H,dv]."""
    q, k = _kda._prepared(q, k, qk_prep)
    return _decode("kda_lina_decode_tokens", q, k, v, log_decay, state, out, 4)

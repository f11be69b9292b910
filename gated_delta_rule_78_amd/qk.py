"""Per-head norm of queries and keys with the position rotation: binding of
``kda_qk_norm_rope`` and its backward.

    y = R(positions x inv_freq) (w + weight_offset) x r

r makes each head's root mean square ("rms") or length ("l2", the unit keys the delta rule
asks for) one, or is 1 (None).  R turns channel pairs by the token's position on one or several
axes.
"""
from __future__ import annotations

import ctypes
import functools

import gated_delta_rule_78_amd as _kda

_NORMS = {None: 0, "none": 0, "rms": 1, "l2": 2}


def rope_inv_freq(rotary_dim, base=10000.0, device="cuda"):
    """base ** (-2 c / rotary_dim), c < rotary_dim / 2, as the float64 tensor qk_norm_rope takes."""
    torch = _kda._torch()
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    c = torch.arange(rotary_dim // 2, dtype=torch.float64)
    return (float(base) ** (-2.0 * c / rotary_dim)).to(device)


def _step(shape, stride, nm):
    """Elements between tokens of [B,T,H,d] or [B,H,d] whose rows of a token are dense."""
    H, d = shape[-2:]
    if 0 in shape:
        return H * d
    if (d > 1 and stride[-1] != 1) or (H > 1 and stride[-2] != d):
        raise ValueError(f"{nm}: the heads of a token must lie back to back")
    step = expect = None
    for n, st in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if n == 1:
            continue
        if step is None:
            step = expect = st
        if st != expect:
            raise ValueError(f"{nm}: tokens must be evenly spaced")
        expect = st * n
    step = H * d if step is None else step
    if step < H * d:
        raise ValueError(f"{nm}: tokens must not overlap")
    return step


@functools.lru_cache(maxsize=1024)
def _shape(q, k, norm, eps, weight_offset, freqs, positions, sections, interleaved):
    """(the C shape, bytes of the backward's workspace) of a call with these sizes, once checked.
    q, k: (shape, stride, dtype) or None; freqs, positions: (shape, dtype) or None."""
    torch = _kda._torch()
    if norm not in _NORMS:
        raise ValueError(f"unknown norm {norm!r}")
    (qs, qt, dtype) = q
    if len(qs) not in (3, 4):
        raise ValueError("q: [B,T,H,d] or [B,H,d]")
    lead, (Hq, d) = tuple(qs[:-2]), qs[-2:]
    if k is not None:
        if k[2] != dtype:
            raise TypeError("k must have the dtype of q")
        if len(k[0]) != len(qs) or tuple(k[0][:-2]) != lead or k[0][-1] != d:
            raise ValueError("shapes: q [..., Hq, d]; k [..., Hk, d]")
    n = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    s = _kda.QkShape(tokens=n, q_heads=Hq, k_heads=0 if k is None else k[0][-2], d=d, norm=_NORMS[norm],
                     eps=eps, weight_offset=weight_offset, interleaved=int(interleaved),
                     dtype=_kda._dtype_code_of(dtype))
    s.q_stride = _step(qs, qt, "q")
    s.k_stride = 0 if k is None else _step(k[0], k[1], "k")
    if (freqs is None) != (positions is None):
        raise ValueError("inv_freq and positions go together")
    if freqs is not None:
        if freqs[1] != torch.float64 or len(freqs[0]) != 1:
            raise TypeError("inv_freq must be a 1-D float64 tensor (rope_inv_freq makes one)")
        if positions[1] not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64")
        half = freqs[0][0]
        sec = [half] if sections is None else sections
        if not 1 <= len(sec) <= 4 or min(sec) < 0 or sum(sec) != half:
            raise ValueError("sections: up to four counts of frequencies that add up to inv_freq's")
        want = lead if sections is None else (len(sec), *lead)
        if tuple(positions[0]) != want:
            raise ValueError(f"positions must have the shape {list(want)}")
        s.rotary_dim, s.n_axes, s.positions_64 = 2 * half, len(sec), int(positions[1] == torch.int64)
        for i, x in enumerate(sec):
            s.sections[i] = x
    elif sections is not None:
        raise ValueError("sections need inv_freq and positions")
    return s, int(_kda.lib().kda_qk_norm_rope_bwd_workspace_size(ctypes.byref(s)))


def _call(q, k, norm, eps, weight_offset, inv_freq, positions, sections, interleaved):
    """_shape of these tensors, which have to be on q's device."""
    dev = q.device
    for x, nm in ((q, "q"), (k, "k")):
        if x is not None and (not x.is_cuda or x.device != dev):
            raise ValueError(f"{nm} must be on {dev}")
    _kda._check((inv_freq, positions), ("inv_freq", "positions"), dev)
    # numbers, not the objects that hold them: a tensor would be found again by its identity
    s, need = _shape((q.shape, q.stride(), q.dtype), None if k is None else (k.shape, k.stride(), k.dtype), norm,
                     float(eps), float(weight_offset), None if inv_freq is None else (inv_freq.shape, inv_freq.dtype),
                     None if positions is None else (positions.shape, positions.dtype),
                     None if sections is None else tuple(map(int, sections)), bool(interleaved))
    return s, need, dev


def _weights(ws, d, dev):
    torch = _kda._torch()
    for w, nm in ws:
        if w is not None and (w.dtype != torch.float32 or w.shape != (d,)):
            raise ValueError(f"{nm} must be float32 [{d}]")
    _kda._check([w for w, _ in ws], [nm for _, nm in ws], dev)


def _like(out, x, nm, dev):
    torch = _kda._torch()
    if x is None:
        return None
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.dtype != x.dtype or out.shape != x.shape:
        raise ValueError(f"{nm} must have the shape and dtype of its input")
    _kda._check((out,), (nm,), dev)
    return out


def qk_norm_rope(q, k=None, *, norm="rms", q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, inv_freq=None,
                 positions=None, sections=None, interleaved=False, q_out=None, k_out=None):
    """Norm and rotate each head of q [B,T,Hq,d] and k [B,T,Hk,d] (or [B,H,d], one token each) in
    one pass; bf16 or fp32, d 64 or 128.  q and k may be slices of one projection's output
    (rows of a token dense, tokens evenly spaced).

    norm: "rms", "l2" or None; q_weight, k_weight fp32 [d] or None, used as w + weight_offset.
    inv_freq: float64 [rotary_dim / 2], rotary_dim a multiple of 16 and at most d (the other
    channels are not turned), or None for no rotation.  positions: int32 or int64 [B,T] (or
    [B]); with sections = (n_0, n_1, ...): [axes,B,T], the first n_0 frequencies turned by axis
    0, and so on.  interleaved: pairs (2c, 2c+1) instead of (c, c + rotary_dim / 2).
    q_out, k_out may be q and k themselves where these are contiguous.  Returns (q', k')."""
    s, _, dev = _call(q, k, norm, eps, weight_offset, inv_freq, positions, sections, interleaved)
    _weights(((q_weight, "q_weight"), (k_weight, "k_weight")), q.shape[-1], dev)
    q_out, k_out = _like(q_out, q, "q_out", dev), _like(k_out, k, "k_out", dev)
    p = _kda._addr
    _kda._launch("kda_qk_norm_rope", dev, ctypes.byref(s), p(q), p(k), p(q_weight), p(k_weight), p(inv_freq),
                 p(positions), p(q_out), p(k_out))
    return q_out, k_out


def qk_norm_rope_bwd(d_q, d_k, q, k=None, *, norm="rms", q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0,
                     inv_freq=None, positions=None, sections=None, interleaved=False, workspace=None):
    """Gradients of qk_norm_rope: d_q, d_k are those of its outputs (contiguous, shape and dtype
    of q, k), the rest its arguments.  Returns (dq, dk, d_q_weight, d_k_weight); the weights'
    gradients are fp32, None where there is no weight."""
    torch = _kda._torch()
    s, need, dev = _call(q, k, norm, eps, weight_offset, inv_freq, positions, sections, interleaved)
    if (d_k is None) != (k is None):
        raise ValueError("d_k and k go together")
    for g, x, nm in ((d_q, q, "d_q"), (d_k, k, "d_k")):
        if x is not None and (g.dtype != x.dtype or g.shape != x.shape):
            raise ValueError(f"{nm} must have the shape and dtype of its input")
    _kda._check((d_q, d_k), ("d_q", "d_k"), dev)
    d = q.shape[-1]
    _weights(((q_weight, "q_weight"), (k_weight, "k_weight")), d, dev)
    gq, gk = _like(None, q, "dq", dev), _like(None, k, "dk", dev)
    gwq = torch.empty_like(q_weight) if q_weight is not None else None
    gwk = torch.empty_like(k_weight) if k_weight is not None else None
    if q_weight is None and k_weight is None:
        need = 0
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _kda._check((workspace,), ("workspace",), dev)
    p = _kda._addr
    _kda._launch("kda_qk_norm_rope_bwd", dev, ctypes.byref(s), p(d_q), p(d_k), p(q), p(k), p(q_weight), p(k_weight),
                 p(inv_freq), p(positions), p(gq), p(gk), p(gwq), p(gwk), p(workspace), nbytes)
    return gq, gk, gwq, gwk

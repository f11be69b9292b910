"""Verification of drafted tokens: binding of ``kda_verify_drafts``.

Draft i of a sequence stands while u_i q_i(x_i) < p_i(x_i); after the n that stand, the next token is
drawn from max(p_n - q_n, 0), or from p_n where no draft is left to refuse.  The tokens that come out
are distributed as the target's own (for random numbers that are uniform and independent).
"""
from __future__ import annotations

import functools

import gated_delta_rule_78_amd as _kda

from .lina import _workspace


@functools.lru_cache(maxsize=1024)
def _sizes(p, drafts, q, u, u_next):
    """(B, K, V, dtype code, bytes of workspace) of a call with these shapes and dtypes, once checked."""
    torch = _kda._torch()
    (ps, dtype), (xs, xt) = p, drafts
    if len(ps) != 3 or len(xs) != 2 or ps[0] != xs[0] or ps[1] != xs[1] + 1 or ps[2] < 1:
        raise ValueError("shapes: target_probs [B,K+1,V], drafts [B,K]")
    code = _kda._dtype_code_of(dtype)
    B, K, V = xs[0], xs[1], ps[2]
    if xt != torch.int32:
        raise TypeError("drafts must be int32")
    if q is not None and q != (torch.Size((B, K, V)), dtype):
        raise ValueError("draft_probs must be [B,K,V] in the dtype of target_probs")
    if u[1] != torch.float32 or u_next[1] != torch.float32:
        raise TypeError("u and u_next must be float32")
    if u[0] != (B, K) or u_next[0] != (B,):
        raise ValueError("shapes: u [B,K], u_next [B]")
    need = int(_kda.lib().kda_verify_drafts_workspace_size(B, K, V, code))
    if need == 0 and B > 0:
        raise ValueError("verify_drafts: too large")
    return B, K, V, code, need


def verify_drafts(target_probs, drafts, draft_probs, u, u_next, workspace=None):
    """How many drafted tokens stand, and the token after them.

    target_probs [B,K+1,V] (bf16 or fp32): the target's probabilities at each draft's place and behind the
    last; drafts int32 [B,K]: an index outside [0, V) ends a sequence's drafts (padding);
    draft_probs [B,K,V] in the dtype of target_probs: the distributions they were drawn from, or None
    where they were chosen outright (all of q on the draft); u fp32 [B,K], u_next fp32 [B]: random numbers
    in [0, 1).  Whether a draft stands is u q < p of these entries as they are (a NaN refuses).  As weights,
    entries that are negative or not finite count nothing; where no weight is left after a
    refusal, the token is drawn from the target's row itself, and it is -1 if that weighs nothing.
    Returns (accepted int32 [B], next_token int32 [B])."""
    torch = _kda._torch()
    B, K, V, code, need = _sizes((target_probs.shape, target_probs.dtype), (drafts.shape, drafts.dtype),
                                 None if draft_probs is None else (draft_probs.shape, draft_probs.dtype),
                                 (u.shape, u.dtype), (u_next.shape, u_next.dtype))
    dev = target_probs.device
    accepted, token = torch.empty((2, B), dtype=torch.int32, device=dev).unbind(0)
    workspace, nbytes = _workspace(need, workspace, dev)
    _kda._check((target_probs, drafts, draft_probs, u, u_next, workspace),
                ("target_probs", "drafts", "draft_probs", "u", "u_next", "workspace"), dev)
    p = _kda._addr
    _kda._launch("kda_verify_drafts", dev, B, K, V, code, p(target_probs), p(drafts), p(draft_probs), p(u), p(u_next),
                 p(accepted), p(token), p(workspace), nbytes)
    return accepted, token

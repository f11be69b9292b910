"""Cases of the linear-attention and query/key preparation operators, with their plain forms.

own = False computes every operator in elementary torch operations (fp32, fp64 for
decay sums and rotation angles); own = True makes the library's calls.

Operators ("op"):
  lina_fwd     S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over whole sequences
  lina_decode  the same for the next token(s) of every sequence, state in place
  lina_bwd     gradients of q, k, v, g and the start state
  qk           per-head norm of q and k and position rotation, one or several axes
  qk_bwd       its gradients
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _lina(name, op, B, T, H, Hk=None, dk=128, dv=128, dtype="bf16", decay="token", seqs=0, states=True):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "Hk": Hk or H, "dk": dk, "dv": dv, "dtype": dtype,
            "decay": decay, "seqs": seqs, "states": states}


def _qk(name, op, B, T, Hq, Hk, d=128, dtype="bf16", norm="rms", rotary=128, axes=1, interleaved=False, weights=True,
        packed=False, far=0):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "dtype": dtype, "norm": norm,
            "rotary": rotary, "axes": axes, "interleaved": interleaved, "weights": weights, "packed": packed, "far": far}


def listed():
    return [
        # one short fp32 prompt of an odd length, where the launches are all the time there is
        _lina("lina_fwd_t130_f32", "lina_fwd", 1, 130, 2, dk=64, dv=64, dtype="f32"),
        # the batched prompt the library's headline is quoted on
        _lina("lina_fwd_b4_t8k", "lina_fwd", 4, 8192, 32),
        # one long document: few heads, a long chain
        _lina("lina_fwd_t128k", "lina_fwd", 1, 131072, 16),
        # a server's prefill batch: ragged prompts packed back to back, q and k shared by four
        # value heads, one fixed decay per head
        _lina("lina_fwd_ragged", "lina_fwd", 1, 20011, 32, Hk=8, decay="head", seqs=24),
        # one user's next token
        _lina("lina_decode_b1", "lina_decode", 1, 1, 32),
        # a full serving batch's next token
        _lina("lina_decode_b256", "lina_decode", 256, 1, 32),
        # a small training step in fp32 with an odd length
        _lina("lina_bwd_t1001_f32", "lina_bwd", 2, 1001, 4, dk=64, dv=64, dtype="f32"),
        # the training step at the headline shape, decay learned per token
        _lina("lina_bwd_b4_t8k", "lina_bwd", 4, 8192, 32),
        # one decode step's queries and keys
        _qk("qk_decode_b8", "qk", 8, 1, 32, 8, packed=True, far=100000),
        # an image / video prompt: three position axes, q and k inside a packed projection
        _qk("qk_axes_32k", "qk", 4, 8192, 32, 8, axes=3, packed=True),
        # L2-normalised q and k for the delta rule, half of the channels rotated, fp32, odd length
        _qk("qk_bwd_t1237_f32", "qk_bwd", 3, 1237, 16, 16, d=64, dtype="f32", norm="l2", rotary=32, interleaved=True,
            weights=False),
        # the training step at the headline shape
        _qk("qk_bwd_32k", "qk_bwd", 4, 8192, 32, 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lina_fwd", "lina_fwd", "lina_decode", "lina_bwd", "lina_bwd", "qk", "qk_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("lina"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        H = min(32, Hk * rng.choice([1, 1, 2, 4]))
        Hk = Hk if H % Hk == 0 else H
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        decay = rng.choice(["token", "token", "head"])
        if op == "lina_decode":
            return _case(_lina("", op, _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 5]), H, Hk, dk, dv, dtype, decay))
        most = (32768 * 32 if dtype == "bf16" else 8192 * 16) // H
        T = min(_log(rng, 1, 131072 if op == "lina_fwd" else 32768), most)
        B = min(_log(rng, 1, 16), max(1, most // T))
        seqs = rng.choice([0, 0, 0, rng.randint(1, 40)])
        if seqs:
            B, T = 1, B * T
        return _case(_lina("", op, B, T, H, Hk, dk, dv, dtype, decay, seqs, rng.random() < 0.6))
    d = rng.choice([64, 128])
    Hq = rng.choice([1, 4, 7, 16, 32])
    Hk = rng.choice([1, 4, 8]) if Hq >= 8 else 1
    most = 32768 if dtype == "bf16" else 8192
    T = _log(rng, 1, 32768)
    T = min(T, most)
    B = min(_log(rng, 1, 64), max(1, most // T))
    return _case(_qk("", op, B, T, Hq, Hk, d, dtype, rng.choice(["rms", "rms", "l2", "none"]),
                     rng.choice([d, d, d // 2, 32]), rng.choice([1, 1, 3]), rng.random() < 0.3, rng.random() < 0.7,
                     op == "qk" and rng.random() < 0.5, rng.choice([0, 0, 1000000])))


def _case(c):
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _sections(case):
    """Frequencies of each axis: a quarter for time, the rest split over height and width."""
    n = case["rotary"] // 2
    if case["axes"] == 1:
        return [n]
    t = n // 4
    h = (n - t + 1) // 2
    return [t, h, n - t - h]


def _offsets(case, seed):
    """Ragged offsets of a packed batch (host list): lengths from zero to several times the mean."""
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    n, T = case["seqs"], case["T"]
    cuts = torch.randint(0, T + 1, (n - 1,), generator=g).sort().values.tolist() if n > 1 else []
    return [0] + cuts + [T]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = _dt(case)

    def randn(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    st = {"case": case}
    if case["op"].startswith("lina"):
        B, T, H, Hk, dk, dv = (case[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))

        def unit(*s):  # rows of unit length, as every caller of the delta rule has them
            x = randn(*s)
            return (x / x.norm(dim=-1, keepdim=True)).to(dt)

        st["q"], st["k"] = unit(B, T, Hk, dk), unit(B, T, Hk, dk)
        st["v"] = randn(B, T, H, dv).to(dt)
        if case["decay"] == "token":  # memories of a few to some hundred tokens, learned per token
            rate = torch.logspace(-2.5, 0, H, device=DEV)
            st["g"] = -rate * torch.nn.functional.softplus(randn(B, T, H))
        else:  # memories of 16 to 2,048 tokens, one for each head
            st["g"] = torch.log1p(-torch.exp2(-torch.linspace(4, 11, H, device=DEV)))
        if case["op"] == "lina_decode":
            if T == 1:
                st["q"], st["k"], st["v"] = st["q"][:, 0].contiguous(), st["k"][:, 0].contiguous(), st["v"][:, 0].contiguous()
                st["g"] = st["g"][:, 0].contiguous() if case["decay"] == "token" else st["g"]
            st["S"] = 0.5 * randn(B, H, dk, dv)
            return st
        st["cu"] = torch.tensor(_offsets(case, seed), dtype=torch.int32, device=DEV) if case["seqs"] else None
        n = case["seqs"] or B
        st["s0"] = 0.5 * randn(n, H, dk, dv) if case["states"] else None
        if case["op"] == "lina_bwd":
            st["d_o"] = randn(B, T, H, dv).to(dt)
            st["d_sT"] = randn(n, H, dk, dv) if case["states"] else None
        return st
    B, T, Hq, Hk, d = (case[n] for n in ("B", "T", "Hq", "Hk", "d"))
    if case["packed"]:  # one projection's output holds q, k and v of each token
        qkv = (2.0 * randn(B, T, Hq + 2 * Hk, d)).to(dt)
        st["q"], st["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    else:
        st["q"], st["k"] = (2.0 * randn(B, T, Hq, d)).to(dt), (2.0 * randn(B, T, Hk, d)).to(dt)
    st["wq"] = 1.0 + 0.2 * randn(d) if case["weights"] else None
    st["wk"] = 1.0 + 0.2 * randn(d) if case["weights"] else None
    n = case["rotary"] // 2
    st["inv"] = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=DEV) / n)
    t = torch.arange(T, device=DEV) + case["far"]
    base = torch.randint(0, 64, (B, 1), generator=gen, device=DEV)
    if case["axes"] == 1:
        st["pos"] = (t[None] + base).to(torch.int32)
    else:  # frames of 24 x 32 patches
        st["pos"] = torch.stack([t // 768 + base, t % 768 // 32 + 0 * base, t % 32 + 0 * base]).to(torch.int32)
    st["sections"] = _sections(case)
    if case["op"] == "qk_bwd":
        st["dq"], st["dk"] = randn(B, T, Hq, d).to(dt), randn(B, T, Hk, d).to(dt)
    return st


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _chunks(st):
    """Token index [N, C] of every chunk, which of them exist, the sequence of each chunk,
    and the number of sequences.  A packed batch has at most T / C + n chunks."""
    case = st["case"]
    B, T = case["B"], case["T"]
    C = 64 if T < 1024 else 256
    col = torch.arange(C, device=DEV)
    if st["cu"] is None:
        per = -(-T // C)
        n = torch.arange(B * per, device=DEV)
        start, seq = (n // per) * T + (n % per) * C, n // per
        end, count = (seq + 1) * T, B
    else:
        cu = st["cu"].long()
        lens = cu[1:] - cu[:-1]
        num = (lens + C - 1) // C
        last = num.cumsum(0)
        N, count = T // C + lens.numel(), lens.numel()
        n = torch.arange(N, device=DEV)
        seq = torch.searchsorted(last, n, right=True)
        some = seq < count
        at = seq.clamp(max=count - 1)
        start = cu[at] + (n - (last - num)[at]) * C
        end = torch.where(some, cu[at + 1], start)
        seq = torch.where(some, at, torch.full_like(at, -1))
    idx = start[:, None] + col
    valid = idx < end[:, None]
    return idx.clamp(max=B * T - 1), valid, seq, count


def _lay(x, idx, valid, groups=1):
    """[B, T, h, d] -> fp32 [h * groups, N, C, d], zeros where no token is."""
    x = x.reshape(-1, x.shape[2], x.shape[3])[idx].float() * valid[..., None, None]
    x = x.permute(2, 0, 1, 3)
    return (x.repeat_interleave(groups, 0) if groups > 1 else x).contiguous()


def _back(x, idx, valid, like, groups=1):
    """The inverse of _lay, summed over shared heads."""
    if groups > 1:
        x = x.reshape(x.shape[0] // groups, groups, *x.shape[1:]).sum(1)
    out = torch.zeros(like.shape[0] * like.shape[1], like.shape[2], like.shape[3], device=DEV)
    out[idx[valid]] = x.permute(1, 2, 0, 3)[valid]
    return out.reshape(like.shape).to(like.dtype)


class _Walk:
    """The chunked form both directions share: decays in fp64, products in fp32."""

    def __init__(self, st):
        case = st["case"]
        B, T, H = case["B"], case["T"], case["H"]
        self.r = H // case["Hk"]
        self.idx, self.valid, self.seq, self.count = _chunks(st)
        g = st["g"].double()
        g = g.expand(B, T, H) if g.dim() == 1 else g
        g = (g.reshape(B * T, H)[self.idx] * self.valid[..., None]).permute(2, 0, 1)
        G = g.cumsum(-1)
        P = G[..., -1].cumsum(-1)                                   # [H, N] decay up to each chunk's end
        P0 = P - G[..., -1]                                         # up to its start
        C = G.shape[-1]
        tri = torch.ones(C, C, dtype=torch.bool, device=DEV).tril()
        self.D = torch.where(tri, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp().float(), 0.0)
        self.row = G.exp().float()[..., None]                       # chunk start -> token
        self.col = (G[..., -1:] - G).exp().float()[..., None]       # token -> chunk end
        self.tot = G[..., -1].exp().float()
        same = (self.seq[:, None] == self.seq[None, :]) & (self.seq[:, None] >= 0)
        N = same.shape[0]
        before = torch.ones(N, N, dtype=torch.bool, device=DEV).tril(-1) & same
        # end of chunk m -> start of chunk n
        self.W = torch.where(before, (P0[:, :, None] - P[:, None, :]).clamp(max=0).exp().float(), 0.0)
        self.of = torch.arange(self.count, device=DEV)[:, None] == self.seq      # [count, N]
        first = torch.where(self.of, torch.arange(N, device=DEV), N).amin(-1).clamp(max=N - 1)
        n = self.seq.clamp(min=0)
        off = P0 - P0[:, first[n]]                                  # sequence start -> chunk start
        whole = (G[..., -1][:, None, :] * self.of).sum(-1)          # [H, count]
        self.length = whole.exp().float()
        self.from0 = (off.exp() * (self.seq >= 0)).float()
        self.to_end = ((whole[:, n] - off - G[..., -1]).clamp(max=0).exp() * (self.seq >= 0)).float()


def _lina_fwd_plain(st):
    case = st["case"]
    w = _Walk(st)
    q, k = (_lay(st[n], w.idx, w.valid, w.r) for n in ("q", "k"))
    v = _lay(st["v"], w.idx, w.valid)
    H, N, C, dk = q.shape
    dv = v.shape[-1]
    Bm = (k * w.col).transpose(2, 3) @ v                                        # [H, N, dk, dv]
    S = (w.W @ Bm.reshape(H, N, dk * dv)).reshape(H, N, dk, dv)
    of = w.of.float()
    sT = torch.einsum("hn,sn,hnx->shx", w.to_end, of, Bm.reshape(H, N, dk * dv)).reshape(w.count, H, dk, dv)
    if st["s0"] is not None:
        s0 = st["s0"].transpose(0, 1)                                           # [H, count, dk, dv]
        S = S + w.from0[..., None, None] * s0[:, w.seq.clamp(min=0)]
        sT = sT + (w.length[..., None, None] * s0).transpose(0, 1)
    o = ((q @ k.transpose(2, 3)) * w.D) @ v + (q * w.row) @ S
    return _back(o, w.idx, w.valid, st["v"]), sT


def _lina_bwd_plain(st):
    case = st["case"]
    w = _Walk(st)
    q, k = (_lay(st[n], w.idx, w.valid, w.r) for n in ("q", "k"))
    v, do = (_lay(st[n], w.idx, w.valid) for n in ("v", "d_o"))
    H, N, C, dk = q.shape
    dv = v.shape[-1]
    n = w.seq.clamp(min=0)
    Bm = (k * w.col).transpose(2, 3) @ v
    S = (w.W @ Bm.reshape(H, N, -1)).reshape(H, N, dk, dv)                      # state at each chunk's start
    Rm = (q * w.row).transpose(2, 3) @ do
    R = (w.W.transpose(1, 2) @ Rm.reshape(H, N, -1)).reshape(H, N, dk, dv)      # its gradient at each chunk's end
    ds0 = torch.einsum("hn,sn,hnx->shx", w.from0, w.of.float(), Rm.reshape(H, N, -1)).reshape(w.count, H, dk, dv)
    if st["s0"] is not None:
        S = S + w.from0[..., None, None] * st["s0"].transpose(0, 1)[:, n]
        d_sT = st["d_sT"].transpose(0, 1)
        R = R + w.to_end[..., None, None] * d_sT[:, n]
        ds0 = ds0 + (w.length[..., None, None] * d_sT).transpose(0, 1)
    A = (q @ k.transpose(2, 3)) * w.D
    E = (do @ v.transpose(2, 3)) * w.D
    a, b = (do @ S.transpose(2, 3)) * w.row, (v @ R.transpose(2, 3)) * w.col
    dq, dk_ = E @ k + a, E.transpose(2, 3) @ q + b
    dv_ = A.transpose(2, 3) @ do + (k * w.col) @ R
    # decays: every path from a token j < t to a token i >= t passes t
    M = (A * (do @ v.transpose(2, 3))).tril(-1)
    a, b = (a * q).sum(-1), (b * k).sum(-1)
    suffix = (M.sum(-1) - M.sum(-2) + a).flip(-1).cumsum(-1).flip(-1)
    dg = suffix + b.cumsum(-1) - b + (w.tot * (R * S).sum((-1, -2)))[..., None]
    dg = _back(dg[..., None], w.idx, w.valid, torch.empty(*st["v"].shape[:3], 1, device=DEV))[..., 0]
    if st["g"].dim() == 1:
        dg = dg.double().sum((0, 1)).float()
    return (_back(dq, w.idx, w.valid, st["q"], w.r), _back(dk_, w.idx, w.valid, st["k"], w.r),
            _back(dv_, w.idx, w.valid, st["v"]), dg, ds0)


def _lina_decode_plain(st):
    case = st["case"]
    r = case["H"] // case["Hk"]
    S, g = st["S"], st["g"]
    tok = st["q"].dim() == 4
    q, k, v = (x if tok else x[:, None] for x in (st["q"], st["k"], st["v"]))
    q, k = (x.float().repeat_interleave(r, 2) for x in (q, k))
    B, T, H, _ = v.shape
    g = g.expand(B, T, H) if g.dim() == 1 else g if tok else g[:, None]
    if T == 1:
        S.mul_(g[:, 0].exp()[..., None, None]).add_(k[:, 0, :, :, None] * v[:, 0, :, None, :].float())
        o = (S * q[:, 0, :, :, None]).sum(2)[:, None]
    else:  # T tokens at once: the state's part and the tokens' own
        G = g.double().cumsum(1).transpose(1, 2)
        D = torch.where(torch.ones(T, T, device=DEV).tril() > 0, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp(),
                        0.0).float()
        qh, kh, vh = (x.float().transpose(1, 2).contiguous() for x in (q, k, v))
        o = ((qh @ kh.transpose(2, 3).contiguous()) * D) @ vh + (qh * G.exp().float()[..., None]) @ S
        o = o.transpose(1, 2)
        S.mul_(G[..., -1].exp().float()[..., None, None])
        S.add_((kh * (G[..., -1:] - G).exp().float()[..., None]).transpose(2, 3).contiguous() @ vh)
    o = o.to(st["v"].dtype)
    return o if tok else o[:, 0], S


def _angles(st):
    """cos and sin [B, T, 1, rotary / 2], the angle in fp64."""
    pos = st["pos"].double()
    if pos.dim() == 3:
        axis = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(st["sections"], device=DEV))
        a = pos[axis].permute(1, 2, 0) * st["inv"]
    else:
        a = pos[..., None] * st["inv"]
    return a.cos().float()[:, :, None], a.sin().float()[:, :, None]


def _rotate(x, cos, sin, interleaved):
    n = cos.shape[-1]
    y, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        u, w = y[..., 0::2], y[..., 1::2]
        y = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = y[..., :n], y[..., n:]
        y = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([y, rest], -1)


def _rms(x, norm):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    s = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((s / x.shape[-1] if norm == "rms" else s) + 1e-6)


def _qk_plain(st):
    case = st["case"]
    cos, sin = _angles(st)

    def one(x, w):
        dt, x = x.dtype, x.float()
        y = x * _rms(x, case["norm"])
        y = y if w is None else y * w
        return _rotate(y, cos, sin, case["interleaved"]).to(dt)

    return one(st["q"], st["wq"]), one(st["k"], st["wk"])


def _qk_bwd_plain(st):
    case = st["case"]
    cos, sin = _angles(st)

    def one(dy, x, w):
        dt, x = x.dtype, x.float()
        z = _rotate(dy.float(), cos, -sin, case["interleaved"])
        r = _rms(x, case["norm"])
        dw = None if w is None else (z * x * r).double().sum((0, 1, 2)).float()
        u = z if w is None else z * w
        if case["norm"] == "none":
            return u.to(dt), dw
        c = (x * u).sum(-1, keepdim=True) * r * r
        return (r * (u - x * (c / x.shape[-1] if case["norm"] == "rms" else c))).to(dt), dw

    (dq, dwq), (dk, dwk) = one(st["dq"], st["q"], st["wq"]), one(st["dk"], st["k"], st["wk"])
    return dq, dk, dwq, dwk


PLAIN = {"lina_fwd": _lina_fwd_plain, "lina_bwd": _lina_bwd_plain, "lina_decode": _lina_decode_plain,
         "qk": _qk_plain, "qk_bwd": _qk_bwd_plain}


def run(state):
    case = state["case"]
    if not own:
        return PLAIN[case["op"]](state)
    import gated_delta_rule_78_amd as kda
    if case["op"] == "lina_fwd":
        return kda.lina_chunk_fwd(state["q"], state["k"], state["v"], state["g"], initial_state=state["s0"],
                                  cu_seqlens=state["cu"])
    if case["op"] == "lina_bwd":
        return kda.lina_chunk_bwd(state["q"], state["k"], state["v"], state["g"], state["d_o"],
                                  initial_state=state["s0"], d_final_state=state["d_sT"], cu_seqlens=state["cu"])
    if case["op"] == "lina_decode":
        call = kda.lina_decode_tokens if state["q"].dim() == 4 else kda.lina_decode_step
        return call(state["q"], state["k"], state["v"], state["g"], state["S"]), state["S"]
    more = dict(norm=case["norm"], q_weight=state["wq"], k_weight=state["wk"], eps=1e-6, inv_freq=state["inv"],
                positions=state["pos"], sections=state["sections"] if case["axes"] > 1 else None,
                interleaved=case["interleaved"])
    if case["op"] == "qk":
        return kda.qk_norm_rope(state["q"], state["k"], **more)
    return kda.qk_norm_rope_bwd(state["dq"], state["dk"], state["q"], state["k"], **more)


# ---------------------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("lina"):
        B, T, H, Hk, dk, dv = (case[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
        rows, n = B * T, case["seqs"] or B
        state = 4 * n * H * dk * dv
        decay = 4 * (rows * H if case["decay"] == "token" else H)
        if case["op"] == "lina_decode":
            return {"bytes": 2 * state + rows * es * (2 * Hk * dk + 2 * H * dv) + decay, "flops": rows * H * 5 * dk * dv}
        qk, vo = rows * Hk * dk * es, rows * H * dv * es
        flops = rows * H * (4 * dk * dv + 64 * (dk + dv))  # chunks of 64: half of a 64 x 64 product twice, state in and out
        if case["op"] == "lina_fwd":
            return {"bytes": 2 * qk + 2 * vo + decay + state * (2 if case["states"] else 1), "flops": flops}
        return {"bytes": 4 * qk + 3 * vo + 2 * decay + state * (3 if case["states"] else 1), "flops": 3 * flops}
    B, T, Hq, Hk, d = (case[n] for n in ("B", "T", "Hq", "Hk", "d"))
    x = B * T * (Hq + Hk) * d
    small = 4 * case["axes"] * B * T + 4 * case["rotary"] + (8 * d if case["weights"] else 0)
    if case["op"] == "qk":
        return {"bytes": 2 * x * es + small, "flops": 8 * x}
    return {"bytes": 3 * x * es + small + (8 * d if case["weights"] else 0), "flops": 16 * x}


def _exact_lina(st):
    """Every output as a sum over pairs of tokens (no states but the first and the last), one
    sequence, one head and one block of rows at a time."""
    case = st["case"]
    B, T, H, Hk, dk, dv = (case[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
    bwd, r, f8 = case["op"] == "lina_bwd", H // Hk, dict(dtype=torch.float64, device=DEV)
    cu = st["cu"].tolist() if st["cu"] is not None else [T * i for i in range(B + 1)]
    flat = {n: st[n].reshape(B * T, -1, st[n].shape[-1]) for n in ("q", "k", "v", "d_o") if n in st}
    g = (st["g"].expand(B * T, H) if st["g"].dim() == 1 else st["g"].reshape(B * T, H)).double()
    o, sT = torch.zeros(B * T, H, dv, **f8), torch.zeros(len(cu) - 1, H, dk, dv, **f8)
    dq, dkk = torch.zeros(B * T, Hk, dk, **f8), torch.zeros(B * T, Hk, dk, **f8)
    dvv, dg, ds0 = torch.zeros(B * T, H, dv, **f8), torch.zeros(B * T, H, **f8), torch.zeros_like(sT)
    for s, (lo, hi) in enumerate(zip(cu, cu[1:])):
        n = hi - lo
        step = max(1, min(n, 1 << 12, (1 << 27) // max(n, 1)))
        for h in range(H):
            q, k = flat["q"][lo:hi, h // r].double(), flat["k"][lo:hi, h // r].double()
            v = flat["v"][lo:hi, h].double()
            L = g[lo:hi, h].cumsum(0)
            S0 = st["s0"][s, h].double() if st["s0"] is not None else torch.zeros(dk, dv, **f8)
            if n == 0:
                sT[s, h] = S0
                if bwd and st["d_sT"] is not None:
                    ds0[s, h] = st["d_sT"][s, h].double()
                continue
            begin, end = L.exp()[:, None], (L[-1] - L).exp()[:, None]
            sT[s, h] = L[-1].exp() * S0 + (k * end).t() @ v
            if bwd:
                do = flat["d_o"][lo:hi, h].double()
                dS = st["d_sT"][s, h].double() if st["d_sT"] is not None else torch.zeros(dk, dv, **f8)
                ds0[s, h] = L[-1].exp() * dS + (q * begin).t() @ do
                a, b = begin * (do @ S0.t()), end * (v @ dS.t())
                dvv[lo:hi, h] += end * (k @ dS)
                dq[lo:hi, h // r] += a
                dkk[lo:hi, h // r] += b
                cross = torch.zeros(n, **f8)
            for i in range(0, n, step):
                e = min(n, i + step)
                seen = torch.arange(e, device=DEV)[None] <= torch.arange(i, e, device=DEV)[:, None]
                D = (L[i:e, None] - L[None, :e]).clamp_(max=0.0).exp_().mul_(seen)
                A = q[i:e] @ k[:e].t()
                if not bwd:
                    o[lo + i:lo + e, h] = A.mul_(D) @ v[:e] + begin[i:e] * (q[i:e] @ S0)
                    continue
                E = do[i:e] @ v[:e].t()
                M = A * E * D
                at = torch.arange(i, e, device=DEV)
                M[at - i, at] = 0.0
                cross[i:e] += M.sum(1)
                cross[:e] -= M.sum(0)
                A, E = A * D, E * D
                dq[lo + i:lo + e, h // r] += E @ k[:e]
                dkk[lo:lo + e, h // r] += E.t() @ q[i:e]
                dvv[lo:lo + e, h] += A.t() @ do[i:e]
            if bwd:
                cross = (cross + (a * q).sum(1)).flip(0).cumsum(0).flip(0)
                through = (b * k).sum(1)
                dg[lo:hi, h] = cross + through.cumsum(0) - through + L[-1].exp() * (S0 * dS).sum()
    if not bwd:
        return o.reshape(st["v"].shape), sT
    dg = dg.sum(0) if st["g"].dim() == 1 else dg.reshape(st["g"].shape)
    return dq.reshape(st["q"].shape), dkk.reshape(st["k"].shape), dvv.reshape(st["v"].shape), dg, ds0


def _exact_decode(st):
    """The recurrence itself, token after token."""
    case = st["case"]
    r, S = case["H"] // case["Hk"], st["S"].double()
    four = st["q"].dim() == 4
    q, k, v = ((x if four else x.unsqueeze(1)).double() for x in (st["q"], st["k"], st["v"]))
    g = st["g"].double()
    out = []
    for t in range(v.shape[1]):
        gt = g if g.dim() == 1 else g[:, t] if four else g
        kt, qt = (torch.repeat_interleave(x[:, t], r, dim=1) for x in (k, q))
        S = torch.exp(gt)[..., None, None] * S + torch.einsum("bhi,bhj->bhij", kt, v[:, t])
        out.append(torch.einsum("bhij,bhi->bhj", S, qt))
    return (torch.stack(out, 1) if four else out[0]), S


def _exact_qk(st):
    """Pairs of channels as complex numbers, turned by exp(i angle)."""
    case = st["case"]
    n = case["rotary"] // 2
    axis = [a for a, c in enumerate(st["sections"]) for _ in range(c)]
    pos = st["pos"].double()
    pos = pos[None] if pos.dim() == 2 else pos
    angle = torch.stack([pos[axis[c]] * st["inv"][c] for c in range(n)], -1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, :, None]

    def pairs(x):
        y = x[..., :2 * n]
        return torch.complex(y[..., 0::2], y[..., 1::2]) if case["interleaved"] else torch.complex(y[..., :n], y[..., n:])

    def channels(z, x):
        y = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)
        return torch.cat([y, x[..., 2 * n:]], -1)

    def scale(x):
        if case["norm"] == "none":
            return torch.ones_like(x[..., :1])
        m = (x * x).mean(-1, keepdim=True) if case["norm"] == "rms" else (x * x).sum(-1, keepdim=True)
        return 1.0 / torch.sqrt(m + 1e-6)

    def forward(x, w):
        x = x.double()
        y = x * scale(x) * (1.0 if w is None else w.double())
        return channels(pairs(y) * turn, y)

    def backward(dy, x, w):
        dy, x = dy.double(), x.double()
        z = channels(pairs(dy) * turn.conj(), dy)
        s = scale(x)
        hat = x * s
        dw = None if w is None else (z * hat).sum((0, 1, 2))
        u = z if w is None else z * w.double()
        if case["norm"] == "none":
            return u, dw
        inner = (u * hat).mean(-1, keepdim=True) if case["norm"] == "rms" else (u * hat).sum(-1, keepdim=True)
        return s * (u - hat * inner), dw

    if case["op"] == "qk":
        return forward(st["q"], st["wq"]), forward(st["k"], st["wk"])
    (dq, dwq), (dk, dwk) = backward(st["dq"], st["q"], st["wq"]), backward(st["dk"], st["k"], st["wk"])
    return dq, dk, dwq, dwk


def exact(case, seed):
    if case["op"] in ("lina_fwd", "lina_bwd"):
        if case["seqs"]:
            cu = _offsets(case, seed)
            pairs = sum((b - a) ** 2 for a, b in zip(cu, cu[1:]))
        else:
            pairs = case["B"] * case["T"] ** 2
        if pairs * case["H"] * (3 if case["op"] == "lina_bwd" else 1) > 3e11 or (case["seqs"] or case["B"]) * case["H"] > 4000:
            return None
        return _exact_lina(prepare(case, seed))
    st = prepare(case, seed)
    return _exact_decode(st) if case["op"] == "lina_decode" else _exact_qk(st)

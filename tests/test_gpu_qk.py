"""Norm and rotation of queries and keys on the GPU against fp64 references (gpu), and the run of
operators they are made for.

Bounds: an output is at most four fp32 products and one sum of two, its row's norm a sum of at most
128 squares (relative 2^-18 at worst in sequence; half of it in the root), angles within 2^-22 of a
turn: |err| <= 2^-17 (|y_c| + |y_pair|); bf16 rounds once more, half a step, 2^-8 of the value.  Gradients have one
more sum over the row: |err| <= 2^-16 (|u| + |x| |x . u|_abs r^2) r.  Weight gradients are fp32 sums of
rows: 2^-22 of the sum of magnitudes per row in the block's share, fp64 above it: 2^-16 of that sum.
"""
import numpy as np
import pytest

import lina_ref as ref

pytestmark = pytest.mark.gpu


def _make(B, T, H, d, dtype, seed, wide=None):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (2.0 * torch.randn(B, T, wide or H, d, generator=g)).to(dt).cuda()
    return x[:, :, :H] if wide else x


def _np(x):
    return x.detach().double().cpu().numpy()


def _setup(B, T, rot, axes, base, seed, p64=False):
    import torch

    import gated_delta_rule_78_amd as kda
    m = rot // 2
    if m == 0:
        return {}, np.zeros((1, B * T), np.int64), np.zeros(0), [0]
    sec = [m] if axes == 1 else [m - 2 * (m // 3), m // 3, m // 3] if axes == 3 else [1, 0, 2, m - 3]
    r = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 5000, (len(sec), B, T), generator=r) + base
    inv = kda.rope_inv_freq(rot)
    p = pos.cuda() if p64 else pos.to(torch.int32).cuda()
    kw = dict(inv_freq=inv, positions=p if axes > 1 else p[0], sections=sec if axes > 1 else None)
    return kw, pos.reshape(len(sec), B * T).numpy(), inv.cpu().numpy(), sec


def _pair(y, m, inter):
    """The other channel of each turned pair (0 elsewhere)."""
    o = np.zeros_like(y)
    if inter:
        o[..., 0:2 * m:2], o[..., 1:2 * m:2] = y[..., 1:2 * m:2], y[..., 0:2 * m:2]
    else:
        o[..., :m], o[..., m:2 * m] = y[..., m:2 * m], y[..., :m]
    return o


CASES = [
    # d, rotary, axes, interleaved, norm, weights, base, int64
    (128, 128, 1, False, "rms", True, 0, False),
    (128, 128, 3, False, "rms", True, 0, True),
    (64, 64, 1, True, "l2", False, 10 ** 6, False),
    (128, 64, 3, True, "rms", True, -2500, True),
    (64, 32, 4, False, "l2", True, 0, False),
    (64, 16, 1, False, None, False, 2 ** 31 - 6000, False),
    (128, 96, 1, False, "rms", False, 0, False),
    (128, 0, 1, False, "l2", True, 0, False),
    (64, 0, 1, False, None, True, 0, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("B,T,Hq,Hk,wide", [(1, 1, 1, 0, 0), (2, 33, 7, 2, 12), (3, 130, 4, 4, 0)])
def test_forward_and_backward(B, T, Hq, Hk, wide, case, dtype):
    import torch

    import gated_delta_rule_78_amd as kda
    d, rot, axes, inter, norm, weights, base, p64 = case
    seed = B * T + d
    q = _make(B, T, Hq, d, dtype, seed, wide)
    k = _make(B, T, Hk, d, dtype, seed + 1, wide) if Hk else None
    r = torch.Generator().manual_seed(seed)
    wq, wk = ((0.2 * torch.randn(d, generator=r)).cuda() if weights else None for _ in range(2))
    wk = wk if Hk else None
    off = 1.0 if weights else 0.0
    kw, pos, inv, sec = _setup(B, T, rot, axes, base, seed, p64)
    more = dict(norm=norm, eps=1e-6, interleaved=inter, q_weight=wq, k_weight=wk, weight_offset=off, **kw)
    oq, ok = kda.qk_norm_rope(q, k, **more)
    dyq = _make(B, T, Hq, d, dtype, seed + 2)
    dyk = _make(B, T, Hk, d, dtype, seed + 3) if Hk else None
    gq, gk, gwq, gwk = kda.qk_norm_rope_bwd(dyq, dyk, q, k, **more)
    assert (ok is None) == (gk is None) == (Hk == 0)
    assert (gwq is None) == (not weights)
    half = 2.0 ** -8 * (1 + 2.0 ** -6) if dtype == "bf16" else 2.0 ** -24
    m = rot // 2
    for x, w, y, dy, g, gw in ((q, wq, oq, dyq, gq, gwq), (k, wk, ok, dyk, gk, gwk)):
        if x is None:
            continue
        flat = lambda t: _np(t).reshape(B * T, -1, d)
        wn = None if w is None else _np(w) + off
        yr = ref.qk_fwd(flat(x), wn, pos, inv, sec, inter, norm, 1e-6)
        lim = 2.0 ** -17 * (np.abs(yr) + np.abs(_pair(yr, m, inter))) * 2 + half * np.abs(yr)
        assert (np.abs(flat(y) - yr) <= lim + 1e-30).all()
        gr, gwr = ref.qk_bwd(flat(dy), flat(x), wn, pos, inv, sec, inter, norm, 1e-6)
        xa, dya, one = np.abs(flat(x)), np.abs(flat(dy)), np.ones(d) if wn is None else np.abs(wn)
        za = dya + _pair(dya, m, inter)
        rn = ref.rnorm(flat(x), norm, 1e-6)
        ua = za * one
        ca = 0.0 if norm is None else (xa * ua).sum(-1, keepdims=True) * rn * rn / (d if norm == "rms" else 1)
        assert (np.abs(flat(g) - gr) <= 2.0 ** -16 * rn * (ua + xa * ca) + half * np.abs(gr) + 1e-30).all()
        if gw is not None:
            assert (np.abs(_np(gw) - gwr) <= 2.0 ** -16 * (za * xa * rn).sum((0, 1)) + 1e-30).all()


def test_weight_gradient_of_many_rows():
    """More rows than one launch's blocks hold at once; summed in a fixed order."""
    import torch

    import gated_delta_rule_78_amd as kda
    B, T, H, d = 2, 9001, 6, 64
    q, dy = _make(B, T, H, d, "f32", 1), _make(B, T, H, d, "f32", 2)
    w = torch.ones(d, device="cuda")
    a = kda.qk_norm_rope_bwd(dy, None, q, q_weight=w)
    b = kda.qk_norm_rope_bwd(dy, None, q, q_weight=w)
    assert torch.equal(a[2], b[2]) and torch.equal(a[0], b[0])
    x, z = q.double(), dy.double()
    hat = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    want = (z * hat).sum((0, 1, 2))
    assert float(((a[2].double() - want).abs() / (z * hat).abs().sum((0, 1, 2))).max()) <= 2.0 ** -20


def test_weight_gradients_without_a_token():
    """No rows: zeros, also with more heads than the parts that the weight gradients are summed from."""
    import torch

    import gated_delta_rule_78_amd as kda
    for H in (2, 5000):
        q, w = torch.empty(1, 0, H, 64, device="cuda"), torch.ones(64, device="cuda")
        _, _, gw, _ = kda.qk_norm_rope_bwd(q, None, q, q_weight=w)
        assert torch.equal(gw, torch.zeros_like(w))


def test_in_place_and_single_tokens():
    import torch

    import gated_delta_rule_78_amd as kda
    q, k = _make(4, 9, 8, 128, "bf16", 1), _make(4, 9, 2, 128, "bf16", 2)
    inv = kda.rope_inv_freq(128)
    pos = torch.arange(9, device="cuda").repeat(4, 1) + 77
    want = kda.qk_norm_rope(q, k, inv_freq=inv, positions=pos)
    one = [kda.qk_norm_rope(q[:, t], k[:, t], inv_freq=inv, positions=pos[:, t].contiguous()) for t in range(9)]
    for i in range(2):
        assert torch.equal(want[i], torch.stack([x[i] for x in one], 1))
    a, b = q.clone(), k.clone()
    got = kda.qk_norm_rope(a, b, inv_freq=inv, positions=pos, q_out=a, k_out=b)
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_rows_are_apart_and_bad_values_stay_in_theirs():
    """A row that is not finite spoils no other row; rows of zeros stay zeros (eps > 0); channels
    that are not turned keep an infinity without a norm."""
    import torch

    import gated_delta_rule_78_amd as kda
    q = _make(2, 20, 3, 64, "f32", 5)
    inv = kda.rope_inv_freq(32)
    pos = torch.arange(20, device="cuda").repeat(2, 1)
    good = kda.qk_norm_rope(q, inv_freq=inv, positions=pos)[0]
    bad = q.clone()
    bad[0, 3, 1, 7] = float("nan")
    bad[1, 4, 2] = 0.0
    y = kda.qk_norm_rope(bad, inv_freq=inv, positions=pos)[0]
    keep = torch.ones(2, 20, 3, dtype=torch.bool, device="cuda")
    keep[0, 3, 1] = keep[1, 4, 2] = False
    assert torch.equal(y[keep], good[keep])
    assert bool(torch.isnan(y[0, 3, 1]).all()) and bool((y[1, 4, 2] == 0).all())
    bad = q.clone()
    bad[0, 0, 0, 50] = float("inf")
    y = kda.qk_norm_rope(bad, norm=None, inv_freq=inv, positions=pos)[0]
    assert y[0, 0, 0, 50] == float("inf") and int((~torch.isfinite(y)).sum()) == 1


def test_strides_it_refuses():
    import torch

    import gated_delta_rule_78_amd as kda
    x = torch.randn(2, 6, 4, 64, device="cuda")
    for bad in (x.transpose(1, 2), x[..., ::2], x[:, :, ::2], x[:, 1:5], x.expand(2, 6, 4, 64)[:, :1].expand(2, 6, 4, 64)):
        if bad.shape[-1] == 64 and bad.stride(-1) == 1 and bad.stride(-2) == 64 and bad.stride(0) == bad.shape[1] * bad.stride(1):
            continue
        with pytest.raises(ValueError):
            kda.qk_norm_rope(bad)
    with pytest.raises(kda.KdaError):
        kda.qk_norm_rope(x[:, :, :3], q_out=None, k=torch.randn(2, 6, 1, 64, device="cuda"),
                         k_out=x[:, :, :1].contiguous(), eps=-1.0)
    with pytest.raises(ValueError):
        kda.qk_norm_rope(x, inv_freq=kda.rope_inv_freq(64), positions=torch.zeros(2, 5, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        kda.qk_norm_rope(x, inv_freq=kda.rope_inv_freq(64).float(), positions=torch.zeros(2, 6, dtype=torch.int32, device="cuda"))


def test_captured_and_replayed():
    import torch

    import gated_delta_rule_78_amd as kda
    q, k = _make(2, 50, 8, 128, "bf16", 1), _make(2, 50, 2, 128, "bf16", 2)
    w = torch.rand(128, device="cuda")
    kw = dict(inv_freq=kda.rope_inv_freq(128), positions=torch.arange(50, device="cuda").repeat(2, 1), q_weight=w,
              k_weight=w)
    work = lambda: [*kda.qk_norm_rope(q, k, **kw), *kda.qk_norm_rope_bwd(q, k, q, k, **kw)]
    want = [x.clone() for x in work()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = work()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    import torch

    import gated_delta_rule_78_amd as kda
    T, H, d = 140000, 124, 128  # more than 2^31 elements
    q = torch.randn(1, T, H, d, device="cuda", dtype=torch.bfloat16)
    assert q.numel() > 2 ** 31
    inv, pos = kda.rope_inv_freq(d), torch.arange(T, device="cuda")[None]
    y = kda.qk_norm_rope(q, inv_freq=inv, positions=pos)[0]
    z = kda.qk_norm_rope(q[:, -9:].contiguous(), inv_freq=inv, positions=pos[:, -9:].contiguous())[0]
    assert torch.equal(y[:, -9:], z)
    g = kda.qk_norm_rope_bwd(y, None, q, inv_freq=inv, positions=pos)[0]
    gz = kda.qk_norm_rope_bwd(z, None, q[:, -9:].contiguous(), inv_freq=inv, positions=pos[:, -9:].contiguous())[0]
    assert torch.equal(g[:, -9:], gz)


def test_rotation_is_sfda_with_constant_phases():
    """KDA without decay on q and k turned by t theta is SFDA with gates e^(i theta): with
    S = R(t theta) S', the update of S' has the turned k and no gate.  Both sides against the fp64
    oracle's SFDA; the gates are rounded to bf16, so phases are quarter turns (exact)."""
    import torch

    import gated_delta_rule_78_amd as kda
    import oracle
    B, T, H, d = 1, 70, 2, 128
    q = _make(B, T, H, d, "bf16", 1)
    k = _make(B, T, H, d, "bf16", 2)
    v = _make(B, T, H, d, "bf16", 3)
    beta = torch.rand(B, T, H, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    kn = kda.qk_norm_rope(k, norm="l2")[0]
    qn = kda.qk_norm_rope(q, norm="l2")[0]
    turns = torch.arange(d // 2) % 4  # quarter turns of pair c per token
    inv = (turns.double() * (np.pi / 2)).cuda()
    pos = torch.arange(T, device="cuda").to(torch.int32).expand(B, T).contiguous()
    # R(theta)^t moves the state forward: the row-side operands turn backwards with it
    qr, kr = kda.qk_norm_rope(qn, kn, norm=None, inv_freq=-inv, positions=pos, interleaved=True)
    o, _ = kda.chunk_fwd(qr, kr, v, torch.ones_like(q), beta)
    c, s = torch.cos(inv.cpu()).round(), torch.sin(inv.cpu()).round()
    lam = torch.stack([c, s], -1).flatten().bfloat16().expand(B, T, H, d).contiguous()
    bits = lambda x: x.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)
    r, _ = oracle.fwd_sfda(bits(qn), bits(kn), bits(v), bits(lam.cuda()), bits(beta))
    x = o.float().cpu().numpy().transpose(0, 2, 1, 3).reshape(B * H, T, d)
    assert np.abs(x - r).max() <= 2e-2 * np.abs(r).max()  # the delta rule's own parity gate


def test_run_of_the_operators():
    """A layer's step as it is used: one projection's q and k prepared, linear attention and the
    delta rule beside it over a prompt, the next tokens decoded, and the gradients back to the
    projection; against the same steps in fp64."""
    import torch

    import gated_delta_rule_78_amd as kda
    B, T, Hq, H, d = 2, 100, 2, 4, 64
    qkv = _make(B, T + 2, 2 * Hq, d, "f32", 7)
    v = _make(B, T + 2, H, d, "f32", 8)
    g = -torch.rand(H, device="cuda")
    inv, pos = kda.rope_inv_freq(32), torch.arange(T + 2, device="cuda").repeat(B, 1)
    kw = dict(norm="l2", inv_freq=inv, positions=pos[:, :T].contiguous())
    q, k = qkv[:, :T, :Hq].contiguous(), qkv[:, :T, Hq:].contiguous()
    qn, kn = kda.qk_norm_rope(q, k, **kw)
    vp = v[:, :T].contiguous()
    o, S = kda.lina_chunk_fwd(qn, kn, vp, g)
    outs = []
    for t in (T, T + 1):
        q1, k1 = kda.qk_norm_rope(qkv[:, t, :Hq], qkv[:, t, Hq:], norm="l2", inv_freq=inv,
                                  positions=pos[:, t].contiguous())
        outs.append(kda.lina_decode_step(q1, k1, v[:, t].contiguous(), g, S))
    n = B * (T + 2)
    p = _np(pos).reshape(1, n)
    prep = lambda x: ref.qk_fwd(_np(x).reshape(n, Hq, d), None, p, _np(inv), [16], False, "l2", 1e-6).reshape(
        B, T + 2, Hq, d)
    rq, rk = prep(qkv[:, :, :Hq]), prep(qkv[:, :, Hq:])
    r, rS = ref.lina_fwd(rq, rk, _np(v), np.broadcast_to(_np(g), (B, T + 2, H)))
    got = _np(torch.cat([o, torch.stack(outs, 1)], 1))
    assert np.abs(got - r).max() <= 2.0 ** -14 * np.abs(r).max()
    assert np.abs(_np(S) - rS).max() <= 2.0 ** -14 * np.abs(rS).max()
    # gradients of sum(o u) to the projection
    u = _make(B, T, H, d, "f32", 9)
    dqn, dkn, _, dg, _ = kda.lina_chunk_bwd(qn, kn, vp, g, u)
    dq, dk, _, _ = kda.qk_norm_rope_bwd(dqn, dkn, q, k, **kw)
    gr = ref.lina_bwd(rq[:, :T], rk[:, :T], _np(vp), np.broadcast_to(_np(g), (B, T, H)), _np(u))
    p = _np(pos[:, :T]).reshape(1, B * T)
    for dy, x, got in ((gr[0], q, dq), (gr[1], k, dk)):
        want = ref.qk_bwd(dy.reshape(B * T, Hq, d), _np(x).reshape(B * T, Hq, d), None, p, _np(inv), [16], False, "l2",
                          1e-6)[0]
        assert np.linalg.norm(_np(got).reshape(want.shape) - want) <= 2.0 ** -18 * np.linalg.norm(want)
    assert np.abs(_np(dg) - gr[3].sum((0, 1))).max() <= 2.0 ** -16 * np.abs(gr[3]).sum()
    # the same keys (bf16, unit) through the delta rule
    qb, kb = qn.bfloat16(), kn.bfloat16()
    one = torch.ones(B, T, Hq, d, device="cuda", dtype=torch.bfloat16)
    beta = torch.full((B, T, Hq), 0.5, device="cuda", dtype=torch.bfloat16)
    od, _ = kda.chunk_fwd(qb, kb, vp[:, :, :Hq].contiguous().bfloat16(), one, beta)
    assert bool(torch.isfinite(od).all())


def test_prepared_on_the_way_in():
    """qk_prep of the forward and decode entry points equals preparing q and k before the call."""
    import torch

    import gated_delta_rule_78_amd as kda
    B, T, H, d = 2, 70, 2, 128
    qkv = _make(B, T, 3 * H, d, "bf16", 3)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:].contiguous()
    prep = dict(norm="l2", inv_freq=kda.rope_inv_freq(64), positions=torch.arange(T, device="cuda").repeat(B, 1))
    qn, kn = kda.qk_norm_rope(q, k, **prep)
    al = torch.rand(B, T, H, d, device="cuda").bfloat16()
    be = torch.rand(B, T, H, device="cuda").bfloat16()
    g = -torch.rand(B, T, H, device="cuda")
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    assert same(kda.chunk_fwd(q, k, v, al, be, qk_prep=prep), kda.chunk_fwd(qn, kn, v, al, be))
    assert same(kda.lina_chunk_fwd(q, k, v, g, qk_prep=prep), kda.lina_chunk_fwd(qn, kn, v, g))
    cu = torch.tensor([0, 50, B * T], dtype=torch.int32, device="cuda")
    flat = lambda x: x.contiguous().reshape(1, B * T, *x.shape[2:])
    one = dict(prep, positions=prep["positions"].reshape(1, B * T))
    a = [flat(x) for x in (q, k, v, al, be)]
    b = [flat(x) for x in (qn, kn, v, al, be)]
    assert same(kda.chunk_fwd_varlen(*a, cu, qk_prep=one), kda.chunk_fwd_varlen(*b, cu))
    S = torch.randn(B, H, d, d, device="cuda")
    t = dict(prep, positions=prep["positions"][:, 5].contiguous())
    at = lambda *xs: [x[:, 5].contiguous() for x in xs]
    s1, s2 = S.clone(), S.clone()
    assert torch.equal(kda.decode_step(*at(q, k, v, al, be), s1, qk_prep=t), kda.decode_step(*at(qn, kn, v, al, be), s2))
    assert torch.equal(s1, s2)
    s1, s2 = S.clone(), S.clone()
    assert torch.equal(kda.lina_decode_step(*at(q, k, v, g), s1, qk_prep=t), kda.lina_decode_step(*at(qn, kn, v, g), s2))
    assert torch.equal(kda.lina_decode_tokens(q, k, v, g, s1, qk_prep=prep), kda.lina_decode_tokens(qn, kn, v, g, s2))
    assert torch.equal(s1, s2)

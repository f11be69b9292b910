"""Linear attention's backward over several groups of kept states, at forced segment lengths and with
whole chains of several chunks, against the fp64 references (gpu); bounds as in test_gpu_lina.

The decay's gradient is taken afresh from two states every so many chunks (a group): token 1,024 and
what follows are the second group of a sequence, whose number in a packed batch depends on where the
sequence starts.  Calls this small are cut into segments by their own rule; KDA_LINA_SEGMENT pins the
chunks of a segment, read once per process, so each length runs in a child process of its own.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import lina_ref as ref
from test_gpu_lina import _check_bwd, _check_fwd, _dev, _inputs, _np, _out, _state

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,decay", [(1100, "token"), (2100, "head")])
def test_second_and_third_group(T, decay, dtype):
    """Two value tiles; dk and dv in one kernel for bf16."""
    _check_bwd(1, T, 1, 1, 128, 128, dtype, decay, seed=T)


@pytest.mark.parametrize("B,T,Hk,H,dk,dv", [(1, 1100, 4, 4, 128, 128), (2, 1001, 4, 4, 64, 64), (1, 2100, 2, 4, 64, 128)])
def test_fp32_decay_gradient_like_the_others(B, T, Hk, H, dk, dv):
    """With fp32 inputs the decay gradient is held to the norm bound of every other fp32 result, 2^-20."""
    import torch

    import gated_delta_rule_78_amd as kda
    q, k, v, _, u = _inputs(B, T, Hk, H, dk, dv, "f32", seed=5)
    # memories of one to some hundred tokens
    noise = torch.randn(B, T, H, generator=torch.Generator().manual_seed(1))
    g = -torch.logspace(-2.5, 0, H) * torch.nn.functional.softplus(noise)
    dg = _np(kda.lina_chunk_bwd(*_dev(q, k, v, g, u))[3])
    want = ref.lina_bwd(*(_np(x) for x in (q, k, v, g, u)))[3]
    assert np.linalg.norm(dg - want) <= 2.0 ** -20 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_decay_gradient_of_decays_under_fp32(dk, dv, dtype):
    """e^g under 2^-126, fp32's least normal number, is zero to the walks: its gradient is exactly zero, from -inf up to
    ln 2^-126 = -87.34."""
    import torch
    T, H = 330, 2
    u = torch.rand(1, T, H, generator=torch.Generator().manual_seed(7))
    g = -0.02 * u
    for i, deep in enumerate((-88.0, -110.0, -360.0, -450.0, -1e30, -float("inf"))):
        g[(u >= 0.02 * i) & (u < 0.02 * (i + 1))] = deep
    out = _check_bwd(1, T, 1, H, dk, dv, dtype, seed=61, g=g)
    dg = out[3].cpu()
    assert bool((dg[g < -87.5] == 0).all()) and bool((dg[g > -1] != 0).all())


# two sequences of more than 1,024 tokens that start off a multiple of 1,024, with an empty one between
CU = [0, 100, 1300, 1300, 2450, 2460]


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("bf16", 128, 64), ("f32", 64, 128), ("f32", 128, 128)])
def test_packed_groups(dtype, dk, dv):
    out = _check_bwd(1, 2470, 1, 2, dk, dv, dtype, cu=CU, seed=31)
    for x in out[:4]:
        assert bool((x[:, CU[-1]:] == 0).all())


def _short_and_long(pieces, gap):
    """Offsets of sequences of 0 to 12 tokens around longer ones of `pieces` tokens."""
    cu = [0]
    for p in pieces:
        for i in range(gap):
            cu.append(cu[-1] + (5 * i) % 13)
        cu.append(cu[-1] + p)
    return cu


# more sequences than end states, and the reverse; both sequences over 1,000 tokens are cut
@pytest.mark.parametrize("gap", [20, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cut_sequences_among_many(dtype, gap):
    """Start and end states of cut sequences have room of their own, whatever lies between them; the state in
    place gives the same."""
    import torch

    import gated_delta_rule_78_amd as kda
    cu, H = _short_and_long((1200, 700, 1101), gap), 2
    T, n = cu[-1] + 3, len(cu) - 1
    _check_bwd(1, T, 1, H, 64, 64, dtype, cu=cu, seed=71)
    q, k, v, g, _ = _inputs(1, T, 1, H, 64, 64, dtype, seed=72)
    S0 = torch.randn(n, H, 64, 64, generator=torch.Generator().manual_seed(3))
    qd, kd, vd, gd, s = _dev(q, k, v, g, S0)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, sT = kda.lina_chunk_fwd(qd, kd, vd, gd, initial_state=s, cu_seqlens=cud)
    o2, s2 = kda.lina_chunk_fwd(qd, kd, vd, gd, initial_state=s, final_state=s, cu_seqlens=cud)
    assert s2 is s and torch.equal(o[:, :cu[-1]], o2[:, :cu[-1]]) and torch.equal(sT, s)
    rs = ref.packed(cu, ref.lina_fwd, *(_np(x) for x in (q, k, v, g)), states=(_np(S0),))
    ra = ref.packed(cu, ref.lina_fwd, *(np.abs(_np(x)) for x in (q, k, v)), _np(g), states=(np.abs(_np(S0)),))
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        _out(o[:, lo:hi], rs[i][0], ra[i][0], dtype, T, f"o of {i}")
        _state(sT[i:i + 1], rs[i][1], ra[i][1], T, f"state of {i}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_whole_chains(dtype):
    """256 chains of four chunks: none is cut."""
    _check_bwd(2, 200, 64, 128, 64, 64, dtype, seed=17)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [100, 150])
def test_chains_around_the_border(H, dtype):
    """100 chains of six chunks are cut both ways, 150 backward only."""
    _check_fwd(1, 330, H // 2, H, 64, 64, dtype, seed=H)
    _check_bwd(1, 330, H // 2, H, 64, 64, dtype, seed=H)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_chain_of_one_head(dtype):
    _check_fwd(1, 8200, 1, 1, 64, 64, dtype, seed=81)
    _check_bwd(1, 8200, 1, 1, 64, 64, dtype, seed=81)


CHILD = r"""
import sys
sys.path[:0] = [{root!r}, {here!r}]
from test_gpu_lina import _check_bwd, _check_fwd
from test_gpu_lina_groups import CU
for dtype, dk, dv in (("bf16", 128, 128), ("bf16", 64, 128), ("f32", 128, 64)):
    print(dtype, dk, dv, flush=True)
    _check_fwd(1, 1100, 1, 2, dk, dv, dtype, seed=51)
    _check_bwd(1, 1100, 1, 1, dk, dv, dtype, seed=52)
    _check_bwd(1, 2470, 1, 1, dk, dv, dtype, cu=CU, seed=53)
print("ok", flush=True)
"""


@pytest.mark.parametrize("L", [1, 5, 1000])
def test_forced_segments(L):
    """Single chunks; segments that end inside a group; chains whole."""
    print(f"linear attention with KDA_LINA_SEGMENT={L} (child process)", flush=True)
    env = dict(os.environ, KDA_LINA_SEGMENT=str(L))
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, here=HERE)], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=110)
    print(r.stdout[-3000:], r.stderr[-3000:], flush=True)
    assert r.returncode == 0 and r.stdout.rstrip().endswith("ok")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_backward_bad_values(dtype, bad):
    """A value that is not finite reaches no gradient that does not depend on it: dq_i takes u_i and the k_j, v_j
    up to i; dk_j takes v_j, dv_j takes k_j, and both the q_i, u_i from j on."""
    import torch

    import gated_delta_rule_78_amd as kda
    T, d = 150, 64
    q, k, v, g, u = _dev(*_inputs(1, T, 1, 1, d, d, dtype, seed=2))
    good = kda.lina_chunk_bwd(q, k, v, g, u)[:3]
    names = ("q", "k", "v", "u")
    # tokens whose dq, dk, dv may not change when x_t is bad
    before, after, but, all_ = (lambda t: slice(0, t)), (lambda t: slice(t + 1, T)), None, (lambda t: slice(0, T))
    clean = {"q": (all_, after, after), "k": (before, all_, but), "v": (before, but, all_), "u": (but, after, after)}
    for t in (5, 63, 100, 149):
        for i, name in enumerate(names):
            x = [y.clone() for y in (q, k, v, u)]
            x[i][:, t, :, 3] = bad
            got = kda.lina_chunk_bwd(x[0], x[1], x[2], g, x[3])[:3]
            for j, where in enumerate(clean[name]):
                keep = [s for s in range(T) if s != t] if where is None else list(range(T))[where(t)]
                a, b = got[j][:, keep].float(), good[j][:, keep].float()
                # another order of the same sums: fp32 roundings, at most one bf16 step after rounding
                lim = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -17) * float(good[j].float().abs().max())
                assert a.numel() == 0 or float((a - b).abs().max()) <= lim, (t, name, "dq dk dv".split()[j])

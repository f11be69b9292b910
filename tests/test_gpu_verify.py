"""Verification of drafted tokens on the GPU against the fp64 reference, index for index (gpu): all sums are
fp64, so that only a random number within about 1e-13 of a border could tell two orders of summation apart."""
import numpy as np
import pytest

import gdr_ref as ref

pytestmark = pytest.mark.gpu


def _case(B, K, V, dtype="f32", seed=0, sure=False, sharp=3.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    logits = sharp * torch.randn(B, K + 1, V, generator=g)
    p = torch.softmax(logits, -1).to(dt)
    q = torch.softmax(logits[:, :K] + torch.randn(B, K, V, generator=g), -1).to(dt)
    x = torch.zeros(B, K, dtype=torch.int32)
    if K:
        x = torch.multinomial(q.reshape(B * K, V).float(), 1, generator=g).reshape(B, K).to(torch.int32)
    return p, x, None if sure else q, torch.rand(B, K, generator=g), torch.rand(B, generator=g)


def _np(x):
    return None if x is None else x.float().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def _check(p, x, q, u, ul):
    import gated_delta_rule_78_amd as kda
    n, t = kda.verify_drafts(*(None if y is None else y.cuda().contiguous() for y in (p, x, q, u, ul)))
    rn, rt = ref.verify(*(_np(y) for y in (p, x, q, u, ul)))
    assert np.array_equal(_np(n), rn) and np.array_equal(_np(t), rt)
    return _np(n), _np(t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (40, 1, 2), (33, 4, 7), (16, 3, 2047), (16, 3, 2048), (8, 2, 2049), (5, 8, 50257), (2, 100, 333)])
def test_against_the_reference(B, K, V, sure, dtype):
    _check(*_case(B, K, V, dtype, B + V, sure))


def test_no_drafts():
    """K = 0: the next token is drawn from the target's row."""
    n, _ = _check(*_case(9, 0, 1000))
    assert (n == 0).all()


@pytest.mark.parametrize("V", [5, 4100])
def test_padding(V):
    """Drafts outside [0, V) end a sequence's drafts; the token is then drawn from the target's row itself."""
    import torch
    p, x, q, u, ul = _case(7, 5, V, seed=2)
    u = torch.zeros_like(u)
    x[0, 0], x[1, 3], x[2, 1], x[3, 4], x[4, 2], x[5] = -1, -5, V, 2 ** 31 - 1, -(2 ** 31), -1
    n, _ = _check(p, x, q, u, ul)
    assert list(n[:6]) == [0, 3, 1, 4, 2, 0] and n[6] == 5


def test_random_numbers_at_the_ends():
    import torch
    p, x, q, u, ul = _case(6, 3, 3000, seed=3)
    for a in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0):
        for b in (0.0, 2.0 ** -30, 1.0 - 2.0 ** -24, 1.0, 3.0, -1.0):
            _check(p, x, q, torch.full_like(u, a), torch.full_like(ul, b))
    n, t = _check(p, x, q, torch.full_like(u, 2.0), torch.full_like(ul, float("nan")))
    assert (t >= 0).all()


def test_a_draft_as_likely_as_the_target_has_it_stands():
    """q == p: every draft stands for u < 1; with u = 1 none does, and nothing is left but the target's row."""
    import torch
    p, x, _, u, ul = _case(4, 3, 500, seed=4)
    q = p[:, :3].clone()
    assert (_check(p, x, q, u, ul)[0] == 3).all()
    n, _ = _check(p, x, q, torch.ones_like(u), ul)
    assert (n == 0).all()


def test_weights_of_nothing():
    """Rows of zeros, negative entries, infinities and NaN weigh nothing; a row without weight gives -1."""
    import torch
    inf, nan = float("inf"), float("nan")
    p, x, q, u, ul = _case(8, 2, 2500, seed=5)
    u = torch.ones_like(u)  # the first draft is refused, unless p is over q
    p[0] = 0.0
    p[1, 0] = -1.0
    p[2, 0, 5:] = 0.0
    p[3, 0, ::3] = nan
    p[4, 0, ::2] = inf
    q[5, 0, ::2] = nan
    q[6, 0] = inf
    p[7, 0] = torch.where(torch.arange(2500) == 2400, 1.0, 0.0)
    n, t = _check(p, x, q, u, ul)
    assert t[0] == -1 and t[7] in (2400, t[7])
    p[1] = -1.0
    assert _check(p, x, q, u, ul)[1][1] == -1


def test_the_last_weight_of_all():
    """One weight in the last tile, one in the first: the index is one of the two, by the random number."""
    import torch
    V = 3 * 2048 + 1
    p = torch.zeros(4, 1, V)
    p[:, 0, 0], p[:, 0, V - 1] = 0.25, 0.75
    ul = torch.tensor([0.0, 0.25 - 2.0 ** -20, 0.25, 1.0 - 2.0 ** -24])
    _, t = _check(p, torch.zeros(4, 0, dtype=torch.int32), None, torch.zeros(4, 0), ul)
    assert list(t) == [0, 0, V - 1, V - 1]


def test_a_captured_round():
    import torch
    import gated_delta_rule_78_amd as kda
    ins = [y.cuda() for y in _case(5, 3, 3000, seed=0)]
    kda.verify_drafts(*ins)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.verify_drafts(*ins)
    for seed in (1, 2, 3):
        new = [y.cuda() for y in _case(5, 3, 3000, seed=seed)]
        want = kda.verify_drafts(*new)
        for a, b in zip(ins, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_round_of_drafting(dtype):
    """Drafted tokens' outputs with the state left alone, their verification, the state over those that stand: as
    the tokens that stand one by one."""
    import torch

    import gated_delta_rule_78_amd as kda
    from test_gpu_gdr import _dev, _inputs
    B, K, H = 6, 4, 4
    x = _dev(*_inputs(B, K + 1, 2, H, 64, 128, dtype, seed=3)[:5])
    S0 = torch.randn(B, H, 64, 128, device="cuda")
    p, drafts, q, u, ul = [y.cuda() for y in _case(B, K, 777, seed=8)]
    u[0], u[1] = 1.0, 0.0  # none of the first's, all of the second's where p is not zero
    S = S0.clone()
    o = kda.gdr_decode_tokens(*x, S, update=False)
    n, token = kda.verify_drafts(p, drafts, q, u, ul)
    kda.gdr_decode_tokens(None, *x[1:], S, counts=n + 1)
    one = S0.clone()
    for t in range(K + 1):
        before = one.clone()
        ot = kda.gdr_decode_step(*(y[:, t].contiguous() for y in x), one)
        stands = (n >= t).view(-1, 1, 1, 1)
        one = torch.where(stands, one, before)
        keep = (n >= t).view(-1, 1, 1).expand_as(ot)
        assert torch.equal(ot[keep], o[:, t][keep])
    assert torch.equal(one, S)
    assert bool((n >= 0).all()) and bool((n <= K).all()) and bool((token >= 0).all()) and len(set(n.tolist())) > 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("B,K,V", [(700, 1, 5 * 2048 + 1), (500, 2, 9 * 2048 - 7), (2100, 1, 3 * 2048 + 5)])
def test_workgroups_of_several_tiles(B, K, V, sure, dtype):
    """Many sequences share the workgroups, so that one goes through several tiles of a row, the last round of them not all
    there: 6 tiles by 2 workgroups, 9 by 4, 4 by one.  Some drafts are padding."""
    import torch
    p, x, q, u, ul = _case(B, K, V, dtype, B + V, sure)
    x[::7, K - 1] = -1
    ul[:4] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.999, 0.5])
    n, t = _check(p, x, q, u, ul)
    assert len(set((t // 2048).tolist())) == -(-V // 2048)  # every tile has been drawn from


def test_the_one_index_that_weighs_anything():
    """A refused draft; of the target's row one index alone weighs anything, in the second tile."""
    import torch
    p, x, q, u, ul = _case(3, 2, 2500, seed=5)
    x[:, 0] = torch.tensor([3, 2399, 2401])
    p[:, 0] = 0.0
    p[:, 0, 2400] = 1.0
    n, t = _check(p, x, q, torch.ones_like(u), ul)
    assert list(n) == [0, 0, 0] and list(t) == [2400] * 3


def test_odd_entries_at_the_drafts():
    """The rule that lets a draft stand takes the entries as they are: u q < p in fp64."""
    import torch
    inf, nan = float("inf"), float("nan")
    rows = [(0.5, inf, 0.5, 1), (0.5, 0.1, -1.0, 1), (0.5, 0.0, -1.0, 1), (0.5, -0.1, -1.0, 1), (0.5, -1.0, 0.5, 0),
            (0.5, 0.9, inf, 0), (0.0, 0.9, inf, 0), (0.5, nan, 0.5, 0), (0.5, 0.5, nan, 0), (0.0, nan, nan, 0), (0.0, 0.0, 0.5, 0),
            (0.5, inf, inf, 0), (nan, 0.5, 0.5, 0)]
    p, x, q, u, ul = _case(len(rows), 1, 300, seed=6)
    for i, (a, px, qx, _) in enumerate(rows):
        u[i, 0], p[i, 0, x[i, 0]], q[i, 0, x[i, 0]] = a, px, qx
    n, _ = _check(p, x, q, u, ul)
    assert list(n) == [r[3] for r in rows]

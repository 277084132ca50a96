"""GPU parity of moe_route_logits at the borders of its 32-bit choice: rows with
no more experts to choose from than are chosen, sums that cancel, scores whose
sum carries the error.  Indices and counts equal oracle/training.py's (float64);
weights as in test_gpu_route_logits.py: (32 + 2D) u, u = 2^-24, D the spread of
a softmax row's logits.
"""
import numpy as np
import pytest
import torch

import fine_grained_moe_gate_b200 as moe
from oracle import training as ot

from gpu_harness import DEV, check_status

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -120


@pytest.fixture(autouse=True)
def _clean_status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    moe.moe_get_last_error()
    yield


def run_route(z, bias, k, o):
    T, E = z.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    counts = torch.full((E,), -7, dtype=torch.int32, device=DEV)
    opts = moe.route_opts(o.score, o.groups, o.top_groups, o.group_top, o.renormalize, o.scale)
    moe.moe_route_logits(z, bias, moe.MoEShape(T, 64, E, k, 128, 0, 128, moe.MOE_BF16), opts, idx, w, counts)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy(), counts.cpu().numpy()


def check_route(z, bias, k, o):
    idx, w, counts = run_route(z, bias, k, o)
    zn = z.cpu().numpy()
    ri, rw, rc, short = ot.route(zn, None if bias is None else bias.cpu().numpy(), k, o)
    wrong = np.flatnonzero((idx != ri).any(axis=1))
    assert len(wrong) == 0, (len(wrong), wrong[:3], idx[wrong[:3]], ri[wrong[:3]])
    assert (counts == rc).all()
    spread = 0.0
    if o.score == "softmax":
        f = np.where(np.isfinite(zn), zn, np.nan)
        spread = (np.nanmax(f, axis=1) - np.nanmin(f, axis=1))[:, None]
    assert (np.abs(w - rw) <= (32 + 2 * spread) * U * np.abs(rw) + TINY * abs(o.scale)).all()
    return short


@pytest.mark.parametrize("T", [3, 9, 40, 131, 600])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_exactly_k_experts_with_equal_values(T, score):
    """As many experts as are chosen, equal values among them (in several lanes of a token at once): all experts, those
    that a mask leaves, those of the kept groups."""
    g = torch.Generator(device=DEV).manual_seed(T)
    for E, k in ((8, 8), (5, 5), (7, 7), (2, 2), (1, 1), (4, 4)):
        for z in (torch.zeros((T, E), device=DEV), torch.full((T, E), -3.0, device=DEV),
                  torch.randint(-1, 2, (T, E), generator=g, device=DEV).float()):
            for bias in (None, torch.full((E,), 0.25, device=DEV)):
                assert not check_route(z, bias, k, ot.Opts(score=score)).any()
    # masked but for k: experts in one lane, in lanes next to each other, in all lanes
    for E, k, left in ((64, 8, range(0, 32, 4)), (64, 8, [0, 1, 2, 3, 32, 33, 34, 35]), (256, 8, [0, 5, 33, 64, 97, 130, 200, 255]),
                       (60, 6, [3, 7, 11, 35, 39, 43]), (256, 8, [0, 1, 2, 3, 32, 33, 34, 35])):
        z = torch.full((T, E), float("-inf"), device=DEV)
        z[:, list(left)] = torch.randint(0, 2, (T, k), generator=g, device=DEV).float()
        z[::2, list(left)] = 0.0
        for bias in (None, torch.full((E,), -0.5, device=DEV)):
            for renorm in (True, False):
                assert not check_route(z, bias, k, ot.Opts(score=score, renormalize=renorm)).any()
    # kept groups of k experts in all
    for groups, per, top, gtop, k in ((8, 8, 1, 1, 8), (8, 8, 1, 2, 8), (8, 4, 2, 2, 8), (6, 3, 2, 1, 6), (4, 1, 3, 1, 3),
                                      (8, 32, 1, 2, 8)):
        z = torch.randint(-1, 1, (T, groups * per), generator=g, device=DEV).float()
        z[::3] = 0.0
        if per > k:  # of the kept group, all but k are masked
            z.view(T, groups, per)[:, :, k:] = float("-inf")
        for bias in (None, torch.full((groups * per,), 0.125, device=DEV)):
            o = ot.Opts(score=score, groups=groups, top_groups=top, group_top=gtop)
            assert not check_route(z, bias, k, o).any()
    check_status()


@pytest.mark.parametrize("big", [0.5, 16.0, 1000.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_values_whose_summands_cancel(score, big):
    """Biases of both signs, one positive in a group: the two best values of every group are about +big and -big, and
    their sums, a few hundredths, lie closer to each other than the summands' 32-bit error."""
    for groups, per, top, k, T in ((8, 32, 4, 8, 2000), (8, 2, 3, 6, 4000), (8, 8, 3, 12, 3000), (16, 8, 5, 8, 3000)):
        E = groups * per
        g = torch.Generator(device=DEV).manual_seed(E + k)
        z = torch.randn((T, E), generator=g, device=DEV) * (0.002 if score == "sigmoid" else 0.05)
        bias = torch.full((groups, per), -big, device=DEV)
        bias[torch.arange(groups), torch.randint(0, per, (groups,), generator=g, device=DEV)] = big
        bias = bias.view(-1)
        o = ot.Opts(score=score, groups=groups, top_groups=top, group_top=2)
        check_route(z, bias, k, o)
        for t in range(0, 160, 8):  # the form of small batches
            check_route(z[t:t + 8].contiguous(), bias, k, o)
        # unequal summands: one group's members far from zero, another's near it
        near = bias.clone()
        near.view(groups, per)[::2] *= 2.0 ** -10
        check_route(z, near, k, o)
    check_status()


def test_group_values_past_the_largest_number():
    """Two forced experts in a group: their 32-bit sum is infinite, the 64-bit one is not."""
    big = torch.finfo(torch.float32).max
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn((300, 64), generator=g, device=DEV)
    bias = torch.zeros(64, device=DEV)
    for place, value in ((0, big), (1, big), (8, big), (9, big * 0.5), (16, big), (24, big * 0.6), (25, big * 0.6),
                         (32, float("inf")), (40, -big)):
        bias[place] = value
    for score in ("sigmoid", "softmax"):
        for top in (1, 2, 3, 4, 5):
            for rows in (z, z[:8].contiguous()):
                check_route(rows, bias, 6, ot.Opts(score=score, groups=8, top_groups=top, group_top=2))
    check_status()


def test_group_values_with_forced_and_masked_members():
    """Biases of the type's largest and lowest value in one group: in 64 bits they cancel, or make the group the last."""
    big = torch.finfo(torch.float32).max
    g = torch.Generator(device=DEV).manual_seed(4)
    z = torch.randn((300, 32), generator=g, device=DEV)
    for pairs in ([(big, -big), (5e36, -big), (0.0, -2e37), (0.0, 0.0)],
                  [(float("inf"), -1e36), (big, 0.0), (big, big), (1e30, -big)],
                  [(-big, -big), (-2e37, -2e37), (-0.5e37, -0.5e37), (2e37, -big)]):
        bias = torch.full((8, 4), -big, device=DEV)
        for i, pair in enumerate(pairs):  # groups 2 i and 2 i + 1
            bias[2 * i, 1:3] = torch.tensor(pair)
            bias[2 * i + 1, :2] = torch.tensor(pair)
        bias = bias.view(-1)
        for score in ("sigmoid", "softmax"):
            for top in range(2, 8):
                for gtop in (1, 2):
                    for rows in (z, z[:8].contiguous()):
                        check_route(rows, bias, 4, ot.Opts(score=score, groups=8, top_groups=top, group_top=gtop))
    check_status()


@pytest.mark.parametrize("depth", [0.5, 2.0, 3.0, 4.3, 5.5])
def test_softmax_with_a_bias_near_the_error_of_its_sum(depth):
    """One large logit beside many equal ones: the error of 1 / sum then weighs most.  Biases set the large score against
    the others' to within -80 .. 80 units of 2^-24, of which 35 may be the 32-bit values' error."""
    E, k = 256, 1
    g = torch.Generator(device=DEV).manual_seed(int(depth * 10))
    for step in range(-80, 81, 4):
        T = 200
        z = torch.full((T, E), -depth, device=DEV)
        z += torch.randn((T, 1), generator=g, device=DEV) + torch.randn((T, E), generator=g, device=DEV) * 1e-7
        z[:, 17] += depth
        s = torch.softmax(z[0].double(), dim=0)
        bias = torch.zeros(E, device=DEV)
        bias[17] = -(s[17] - s[40] + step * 2.0 ** -24 * s[17]).float()
        check_route(z, bias, k, ot.Opts(score="softmax"))
        check_route(z[:8].contiguous(), bias, k, ot.Opts(score="softmax", groups=2, top_groups=1, group_top=2))
    check_status()


@pytest.mark.parametrize("T,d,E,k", [(130, 64, 64, 6), (700, 256, 160, 6), (2500, 64, 256, 8), (6000, 128, 256, 8), (3000, 64, 256, 12)])
def test_each_replay_sees_its_own_inputs(T, d, E, k):
    """Gate logits, routing and its gradient in one graph: replays on changing tokens and biases, one behind the other,
    give what the same calls give with a synchronisation after each."""
    g = torch.Generator(device=DEV).manual_seed(T)
    sh = moe.MoEShape(T, d, E, k, 128, 0, 128, moe.MOE_BF16)
    co = moe.route_opts(groups=4, top_groups=2, group_top=2)
    n = 8
    xs = torch.randn((n, T, d), generator=g, device=DEV).bfloat16()
    bs = (torch.rand((n, E), generator=g, device=DEV) - 0.5) * 0.1
    wg = (torch.randn((E, d), generator=g, device=DEV) * 0.05).bfloat16()
    dw = torch.randn((T, k), generator=g, device=DEV)
    x, bias, z, dz = xs[0].clone(), bs[0].clone(), torch.empty((T, E), device=DEV), torch.empty((T, E), device=DEV)
    idx, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    counts = torch.empty(E, dtype=torch.int32, device=DEV)
    steps = [lambda: moe.moe_gate_logits(x, wg, sh, z), lambda: moe.moe_route_logits(z, bias, sh, co, idx, w, counts),
             lambda: moe.moe_route_logits_backward(z, idx, dw, None, sh, co, dz)]
    out = (z, idx, w, counts, dz)
    want = []
    for i in range(n):
        x.copy_(xs[i])
        bias.copy_(bs[i])
        for step in steps:
            step()
            torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for step in steps:
            step()
    for rounds in range(3):
        got = []
        for i in range(n):
            x.copy_(xs[i])
            bias.copy_(bs[i])
            graph.replay()
            got.append([t.clone() for t in out])
        torch.cuda.synchronize()
        for i in range(n):
            for a, b in zip(got[i], want[i]):
                assert torch.equal(a, b), (rounds, i)
    check_status()

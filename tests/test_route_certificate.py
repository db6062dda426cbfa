"""Choices of moe_route_scored that float keys get wrong: the ids have to be those of the 64-bit
keys all the same, and equal keys go to the lower expert.

The rows are built so that an expert ranked below the ones next to the border by its float key
has the larger 64-bit key: its score is large and its bias negative, so that its float key is
off by more than theirs, or its key equals theirs in float alone.
"""

import numpy as np
import pytest
import torch

import mixture_experts_layer_04_gb300 as moe
from tests.test_route_scored import check, gen

SCORES = [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID]
F32 = np.float32


def border_rows(T, triples, score, seed):
    """Row t holds three experts A, B and X of triple t % triples; the others are masked (but
    for expert E - 1, which only takes its share of the softmax).  With 64-bit keys
    X > A > B, 6e-9 and 4e-9 apart; A and B have scores under 1e-6 and a bias of 1e-3, X a score
    of about 0.9 and a bias that brings it back to 1e-3."""
    rng = np.random.default_rng(seed)
    E = 3 * triples + 1
    place = rng.permutation(E - 1)
    logits = np.full((T, E), -np.inf)
    bias = np.zeros(E, F32)
    s_x = rng.uniform(0.86, 0.95, triples)
    a, b, x = place[0::3], place[1::3], place[2::3]
    bias[a], bias[b] = F32(1e-3), F32(1e-3)
    bias[x] = (1e-3 - s_x).astype(F32)
    bias[E - 1] = -5.0
    logits[:, E - 1] = 0.0
    for t in range(T):
        i = t % triples
        goal = 1e-3 + rng.uniform(2e-7, 9e-7) - float(bias[x[i]])  # X's score
        lx = float(F32(np.log(goal / (1.0 - goal))))
        if score == moe.SCORE_SIGMOID:
            sx = 1.0 / (1.0 + np.exp(-lx))
            unit = lambda s: np.log(s / (1.0 - s))
        else:  # A's and B's shares of the softmax, low - 6e-9 and low - 10e-9, counted in its sum
            p, q = np.exp(lx) / (1.0 + np.exp(lx)), 16e-9
            low = (p * (1.0 + q) + float(bias[x[i]]) - float(F32(1e-3))) / (1.0 + 2.0 * p)
            total = (1.0 + np.exp(lx)) / (1.0 - 2.0 * low + q)
            sx = np.exp(lx) / total
            unit = lambda s: np.log(s * total)
        low = sx + float(bias[x[i]]) - float(F32(1e-3))
        logits[t, x[i]] = lx
        logits[t, a[i]] = unit(low - 6e-9)
        logits[t, b[i]] = unit(low - 10e-9)
    return torch.tensor(logits, dtype=torch.float32, device="cuda"), torch.tensor(bias, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("triples", [1, 10, 80, 330])
def test_large_scores_with_negative_biases_next_to_small_ones(triples, score):
    T = 2000
    logits, bias = border_rows(T, triples, score, triples)
    E = logits.shape[1]
    for K in (1, 2, 3):
        check(moe.RouteConfig.make(T, E, K, 1, 1, 1, score), logits, bias)


def tied_rows(T, E, dtype, seed, top=1.0):
    """Rows with two to five equal logits at low ids, and one expert of a higher id that is one
    step of the type above them; everything else is clearly below."""
    rng = np.random.default_rng(seed)
    L = torch.full((T, E), 0.0)
    L += torch.tensor(rng.uniform(top - 6.0, top - 2.0, (T, E)), dtype=torch.float32)
    L = L.to(dtype)
    v = torch.tensor(top, dtype=dtype)
    up = torch.tensor(top * (1 + torch.finfo(dtype).eps), dtype=dtype)
    for t in range(T):
        n = int(rng.integers(2, 6))
        at = np.sort(rng.choice(E, n + 1, replace=False))
        L[t, at[:n]] = v
        L[t, at[n]] = up
    return L.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E", [20, 60, 256, 1000])
def test_ties_at_the_border_with_a_better_expert_further_down(E, score):
    # 1: without a bias a step of the logits is lost in the order's low bits; 20: the logistic
    # function is 1 in float (and 6e-10 apart in 64 bits)
    T = 300
    for dtype, code in ((torch.float32, moe.F32), (torch.bfloat16, moe.BF16)):
        for top in (1.0, 20.0):
            logits = tied_rows(T, E, dtype, E, top)
            for bias in (None, torch.zeros(E, device="cuda"),
                         torch.full((E,), 0.25, device="cuda")):
                for K in (1, 2, 3, 5):
                    check(moe.RouteConfig.make(T, E, K, 1, 1, 1, score, dtype=code), logits, bias)


@pytest.mark.gpu
def test_three_saturated_scores():
    logits = torch.tensor([[20.0, 20.0, 21.0]], device="cuda")
    for bias in (None, torch.zeros(3, device="cuda")):
        ids, _ = check(moe.RouteConfig.make(1, 3, 1, score=moe.SCORE_SIGMOID), logits, bias)
        assert ids.item() == 2
    # 64 bits cannot tell 40 from 41 either: the lower id, whichever its logit
    logits = torch.tensor([[39.5, 41.0, 41.0]], device="cuda")
    ids, _ = check(moe.RouteConfig.make(1, 3, 1, score=moe.SCORE_SIGMOID), logits)
    assert ids.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("score", SCORES)
def test_grouped_choices_with_ties_and_better_experts(score):
    T, E = 300, 256
    for top in (1.0, 20.0):
        logits = tied_rows(T, E, torch.float32, 7, top)
        for bias in (None, torch.zeros(E, device="cuda")):
            check(moe.RouteConfig.make(T, E, 2, 8, 4, 2, score), logits, bias)
            check(moe.RouteConfig.make(T, E, 3, 32, 20, 1, score), logits, bias)

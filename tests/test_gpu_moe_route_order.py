"""Without a bias the experts of the groups that stay go by their logits, also where
their scores are equal numbers in 64 bits (sigmoids next to one, softmaxes of zero).
What is expected is written down here, not taken from the oracle: the groups that stay
are plain by construction, and within them it is the order of (logit, index)."""
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs

pytestmark = pytest.mark.gpu


def _expect(x, k, size, kept):
    """ids of each row's k largest logits among the experts of its groups, by sorting."""
    out = []
    for row, groups in zip(x, kept):
        on = sorted((e for e in range(len(row)) if e // size in groups and row[e] > -math.inf), key=lambda e: (-row[e], e))
        out.append((on + [-1] * k)[:k])
    return np.array(out)


@pytest.mark.parametrize("logits,sigmoid,want", [
    ([40.0, 41.0, 42.0, 1.0, 0.0, 0.0, 0.0, 0.0], True, [2, 1, 0, 3]),
    ([0.0, -1.0, -2.0, 1.0, 38.0, 40.0, 39.0, 40.0], True, [5, 7, 6, 4]),
    ([0.5, 0.0, -900.0, -800.0, -1.0, -1.0, -2.0, -math.inf], False, [0, 1, 3, 2]),
    ([-1.0, -1.0, -2.0, -3.0, -801.0, 1.0, 0.0, -800.0], False, [5, 6, 7, 4]),
])
@pytest.mark.parametrize("T", [1, 5, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_by_hand(logits, sigmoid, want, T, dtype):
    if dtype == torch.bfloat16 and -801.0 in logits:
        want = [5, 6, 4, 7]                    # bf16 holds -801 as -800 (a step is 4 there): two equal logits, by index
    x = torch.tensor([logits] * T).to(dtype).cuda()
    for top in (1, 2):
        for k in (1, 2, 4):
            ids, _ = bs.moe_route(x, k, score=int(sigmoid), groups=2, topk_groups=1, group_top=top)
            assert (ids.cpu().numpy() == np.array(want[:k])).all(), (top, k, ids[0].tolist())


CASES = [   # T, E, k, groups, topk_groups: groups of whole lanes, others, more than 512 experts; many tokens
    (40, 8, 3, 2, 1), (40, 64, 6, 4, 2), (40, 256, 8, 8, 4), (40, 512, 10, 16, 4), (40, 160, 6, 8, 3), (24, 1024, 8, 8, 3),
    (40, 128, 16, 64, 9), (4099, 64, 6, 4, 2), (4099, 128, 8, 16, 5), (4099, 256, 8, 8, 4), (4099, 256, 5, 2, 1),
    (4099, 160, 6, 8, 3),
]


@pytest.mark.parametrize("T,E,k,groups,keep", CASES)
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["far", "next", "equal"])
def test_within_the_groups_that_stay(T, E, k, groups, keep, sigmoid, dtype, kind):
    """`keep` groups of each row hold large logits (sigmoid: all of score 1; softmax: two near
    the largest and the rest of score 0), the other groups far smaller ones."""
    g = np.random.default_rng(E + T)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    size, rows = E // groups, 40
    x = np.empty((rows, E))
    kept = [set(g.permutation(groups)[:keep].tolist()) for _ in range(rows)]
    step = {"far": 0.5, "next": 2.0 ** -18 if dtype == "fp32" else 0.25, "equal": 0.0}[kind]   # (an ulp of fp32 at 40 or 2)
    for r in range(rows):
        if sigmoid:
            x[r] = -5.0 - g.random(E)
            base = 40.0
        else:
            x[r] = -3000.0 - g.integers(0, 8, E) * 16.0
            base = -900.0
        for q in kept[r]:
            at = q * size + np.arange(size)
            x[r, at] = base + g.integers(0, 12, size) * step * (1.0 if sigmoid else 32.0)
            if not sigmoid:
                x[r, at[g.permutation(size)[:2]]] = 0.0     # two equal ones: the group's sum
    x = torch.tensor(x).to(t)
    want = _expect(x.double().numpy(), k, size, kept)
    row = g.integers(0, rows, T)
    ids, _ = bs.moe_route(x[torch.from_numpy(row)].cuda(), k, score=int(sigmoid), groups=groups, topk_groups=keep, group_top=2)
    bad = np.argwhere((ids.cpu().numpy() != want[row]).any(1))
    assert not len(bad), (len(bad), ids[int(bad[0, 0])].tolist(), want[row[bad[0, 0]]].tolist())

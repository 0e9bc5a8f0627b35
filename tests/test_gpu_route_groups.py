"""Groups of experts whose values lie near each other or past fp32's range, or are equal in 64 bits although their
logits are not, against the 64-bit definition."""

import math

import numpy as np
import pytest

import fusion_backend_gb300 as fb
from test_gpu_route import check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SCORES = [fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID]


def pinned(E, groups, size, g):
    """A bias of +size for one expert of every group and of -size for the others (size: one number, or one a group)."""
    gs = E // groups
    size = torch.as_tensor(size, dtype=torch.float32).expand(groups)
    bias = -size.repeat_interleave(gs)
    at = torch.arange(groups) * gs + torch.randint(0, gs, (groups,), generator=g)
    bias[at] = size
    return bias.cuda()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("size", [4.0, 16.0, 1000.0, 1e4])
@pytest.mark.parametrize("steps", [1, 8, 64])
def test_sums_of_two_that_cancel(score, size, steps):
    """c of a group's two best is about +size and -size: their sum keeps what fp32 rounds away of each."""
    g = torch.Generator().manual_seed(int(size) + steps)
    E, groups = 64, 8
    # scores of an expert in a group differ by some `steps` of fp32 at `size`
    spread = steps * size * 2.0**-23 * (E if score == fb.SCORE_SOFTMAX else 4)
    lg = (torch.randn(200, E, generator=g) * min(spread, 2.0)).cuda()
    check(lg, 6, pinned(E, groups, size, g), score, groups, 4, fb.GROUP_TOP2)


@pytest.mark.parametrize("score", SCORES)
def test_groups_of_very_different_magnitudes(score):
    """A group far from the cut in the order of the rounded sums, and within its own rounding of it."""
    g = torch.Generator().manual_seed(3)
    size = [0.0, 1e5, 3.0, 1e6, 0.0, 1e3, 30.0, 1e6]
    for E in (64, 256):
        lg = (torch.randn(200, E, generator=g) * 0.3).cuda()
        for top_groups in (1, 3, 5, 7):
            check(lg, 5, pinned(E, 8, size, g), score, 8, top_groups, fb.GROUP_TOP2)
            check(lg, 5, pinned(E, 8, size, g), score, 8, top_groups, fb.GROUP_MAX)


@pytest.mark.parametrize("score", SCORES)
def test_sums_of_two_past_fp32(score):
    g = torch.Generator().manual_seed(5)
    lg = torch.randn(20, 32, generator=g).cuda()
    low = torch.finfo(torch.float32).min
    # a masked group before groups held back by the type's lowest value: they come before it all the same
    bias = torch.zeros(32, device="cuda")
    bias[:8] = -math.inf
    bias[8:16] = low
    bias[24:] = low
    got, _ = check(lg, 12, bias, score, 4, 2, fb.GROUP_TOP2)
    assert (got >= 8).all()
    # sums above the largest number keep their order
    for values in ([3.0e38, 3.4e38, 3.2e38, 1.0], [1.0, 3.4e38, math.inf, 3.0e38], [-3.0e38, -3.4e38, -2.0e38, -math.inf]):
        bias = torch.tensor(values, device="cuda").repeat_interleave(8)
        for top_groups in (1, 2, 3):
            check(lg, 5, bias, score, 4, top_groups, fb.GROUP_TOP2)


def both(lg, k, score, groups, top_groups):
    """Without a bias and with one of zeros: one definition, one answer."""
    a, _ = check(lg, k, None, score, groups, top_groups, fb.GROUP_MAX)
    b, _ = check(lg, k, torch.zeros(lg.shape[1], device="cuda"), score, groups, top_groups, fb.GROUP_MAX)
    assert np.array_equal(a, b)


def test_group_maxima_of_equal_scores():
    """Logits that differ where the scores in 64 bits do not: equal values of groups go to the lower group."""
    lg = torch.full((6, 16), -1.0, device="cuda")
    lg[0, 3], lg[0, 9] = 40.0, 45.0           # sigmoid: 1 in 64 bits
    lg[1] = -800.0
    lg[1, 14] = -760.0                        # 0 in 64 bits
    lg[2, :] = -5.0
    lg[2, 6], lg[2, 11] = 0.0, 1e-20          # 1/2 (softmax: the same power)
    lg[3, 0::4] = torch.tensor([50.0, 60.0, 55.0, 40.0], device="cuda")
    lg[4] = -2000.0
    lg[4, 12], lg[4, 4], lg[4, 8] = 0.0, -900.0, -800.0   # softmax: 1, 0, 0
    lg[5, :] = -math.inf
    lg[5, 9], lg[5, 2] = 90.0, 80.0
    for score in SCORES:
        for groups, top_groups in ((2, 1), (4, 1), (4, 2), (4, 3), (8, 3)):
            both(lg, 2, score, groups, top_groups)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_group_maxima_of_many_rows(score, dtype):
    """Rows drawn from few values, so that groups are equal in the logit, in the score alone, or in neither."""
    g = torch.Generator().manual_seed(7)
    values = torch.tensor([-3000.0, -800.0, -60.0, -2.0, 0.0, 1e-20, 0.5, 3.0, 14.0, 18.0, 40.0, 48.0])
    for E, groups in ((32, 8), (96, 4), (128, 32)):
        # mostly low values, so that the maxima of groups spread over all of them
        at = (torch.rand(300, E, generator=g) ** (E / groups / 2) * len(values)).long().clamp(max=len(values) - 1)
        for top_groups in (1, groups // 2, groups - 1):
            both(values[at].to(dtype).cuda(), 2, score, groups, top_groups)
    lg = torch.randn(500, 64, generator=g).to(dtype).cuda()
    both(lg, 4, score, 8, 3)

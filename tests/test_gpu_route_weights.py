"""Renormalised weights of chosen logits that are all far below 0, and far from each other."""

import pytest

import fusion_backend_gb300 as fb
from test_gpu_route import check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("score", [fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ratios_of_small_scores(score, dtype):
    g = torch.Generator().manual_seed(2)
    # the largest logit from 20 down to -300, the others up to 86 below it
    top = torch.linspace(20, -300, 321)[:, None]
    lg = (top - torch.rand(321, 12, generator=g) * 86).to(dtype)
    lg[:, 3] = top[:, 0].to(dtype)
    for k in (1, 2, 5, 12):
        check(lg.cuda(), k, None, score)
        check(lg.cuda(), k, torch.zeros(12, device="cuda"), score, scale=2.5)
    check(torch.tensor([[-50.0, -95.0, -59.0, -110.0]], dtype=dtype, device="cuda"), 4, None, score)

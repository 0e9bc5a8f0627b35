"""As many rows as the argument blocks can say."""

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = 2**31 - 1


def test_route_of_the_most_tokens():
    lg = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    lg[-1] = -float("inf")
    ids, w = torch.full((T, 1), 7, dtype=torch.int32, device="cuda"), torch.zeros(T, 1, device="cuda")
    fb.moe_ffn_route(lg, 1, scale=0.5, ids=ids, weights=w)
    torch.cuda.synchronize()
    assert int(ids[-1]) == -1 and float(w[-1]) == 0
    assert bool((ids[:-1] == 0).all()) and bool((w[:-1] == 0.5).all())


def test_norm_of_the_most_rows():
    res = torch.full((T, 1), -3.0, dtype=torch.bfloat16, device="cuda")
    res[-1] = 0
    _, n = fb.moe_ffn_norm_residual(res, norm_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert float(n[-1]) == 0 and bool((n[:-1] == -1).all())

"""The operators together, as examples/serving_block.py runs them, against the block's formula in 64 bits."""

import importlib.util
import os

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("serving_block", os.path.join(ROOT, "examples", "serving_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod.ServingBlock(3)


def rms(v):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)


def ffn(x, w):
    g, u = x @ w[0].T, x @ w[1].T
    return (g * torch.sigmoid(g) * u) @ w[2]


def reference(b, residual, normed, adapters, ids):
    """The block in 64 bits for the chosen ids; also each token's c of its choice and of the best expert left out."""
    n, T = normed.double(), residual.shape[0]
    s = torch.sigmoid((normed.float() @ b.router_w.float().T).double())
    c = s + b.bias.double()
    by = c.view(T, b.GROUPS, -1).topk(2, dim=2).values.sum(2)
    kept = torch.zeros_like(by, dtype=torch.bool).scatter_(1, by.topk(b.TOP_GROUPS, dim=1).indices, True)
    c = torch.where(kept.repeat_interleave(b.E // b.GROUPS, 1), c, torch.full_like(c, -1.0))
    top = c.topk(b.TOP_K, dim=1).indices
    assert torch.equal(top.sort(1).values, ids.long().sort(1).values)
    w = s.gather(1, ids.long())
    w = w / w.sum(1, keepdim=True)
    f = ffn(n, b.shexp_w.double())
    for e in range(b.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            f.index_add_(0, t, w[t, j][:, None] * ffn(n[t], b.expert_w[e].double()))
    for t in range(T):
        a = int(adapters[t])
        if a >= 0:
            f[t] += b.lora_scale[a].double() * (b.lora_b[a].double() @ (b.lora_a[a].double() @ n[t]))
    r = residual.double() + rms(f) * b.post_w.double() * b.gate.double()
    return r, rms(r) * b.pre_w.double()


@pytest.mark.parametrize("T", [1, 5, 64])
def test_block(block, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    residual = torch.randn(T, block.H, generator=g, device="cuda")
    _, normed = fb.moe_ffn_norm_residual(residual, w_pre=block.pre_w)
    adapters = torch.randint(-1, block.ADAPTERS, (T,), generator=g, device="cuda", dtype=torch.int32)
    r0, n0 = residual.clone(), normed.clone()
    got_r, got_n = block(residual, normed, adapters)
    assert got_r is residual and got_n is normed
    torch.cuda.synchronize()
    want_r, want_n = reference(block, r0, n0, adapters, block.kept[T]["ids"])
    # the layer's bar (1e-2 rms of its output, which the post norm brings to 1) for the residual; the next norm adds
    # its rounding to bf16
    assert float((residual.double() - want_r).abs().max()) <= 1e-2 * float((want_r - r0.double()).square().mean().sqrt()) + 1e-5
    assert float((normed.double() - want_n).abs().max()) <= 2e-2 * float(want_n.square().mean().sqrt()) + 2.0**-8 * float(want_n.abs().max())
    assert block.kept[T]["layer"].status() == 0


def test_block_in_a_graph(block):
    T = 2
    g = torch.Generator(device="cuda").manual_seed(9)
    residual = torch.randn(T, block.H, generator=g, device="cuda")
    _, normed = fb.moe_ffn_norm_residual(residual, w_pre=block.pre_w)
    adapters = torch.tensor([3, -1], dtype=torch.int32, device="cuda")
    r0, n0 = residual.clone(), normed.clone()
    block(residual, normed, adapters)
    want = residual.clone(), normed.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(residual, normed, adapters)
    for _ in range(2):
        residual.copy_(r0)
        normed.copy_(n0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(residual, want[0]) and torch.equal(normed, want[1])

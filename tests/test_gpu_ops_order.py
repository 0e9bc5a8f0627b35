"""Weights that an operator around the layer writes right before the layer's call read as written: the row kernel
starts its copies of them ahead of its wait on the kernel before it."""

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

H, E, K, I, IS = 2048, 16, 4, 64, 256


class Layer:
    def __init__(self, T, given):
        g = torch.Generator(device="cuda").manual_seed(T)
        self.bf = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.02).bfloat16()
        self.x, self.router, self.expert = self.bf(T, H) * 50, self.bf(E, H), self.bf(E * 3 * I, H)
        self.m = fb.MoeFFN(fb.Shapes(T, H, E, K, I, IS), fb.ACT_BF16, fb.W_BF16)
        self.ids = torch.arange(T * K, device="cuda", dtype=torch.int32).view(T, K) % E if given else None
        self.w = torch.rand(T, K, generator=g, device="cuda")
        self.out = torch.zeros(T, H, device="cuda")

    def __call__(self, shared, gate):
        if self.ids is None:
            self.m(self.x, self.router, self.expert, shared, gate, out=self.out)
        else:
            self.m.routed(self.x, self.ids, self.w, self.expert, shared, gate, out=self.out)
        return self.out


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("writer", ["norm", "adapters"])
def test_weights_written_right_before_the_layer(T, given, writer):
    layer = Layer(T, given)
    rows, n = 3 * IS, 6
    sources, gates = [layer.bf(rows, H) for _ in range(n)], [layer.bf(1, H) for _ in range(n)]
    shared, gate = torch.zeros_like(sources[0]), torch.zeros_like(gates[0])
    a, b, ids = layer.bf(1, 16, H), layer.bf(1, H, 16), torch.zeros(rows, dtype=torch.int32, device="cuda")
    scale = torch.full((H,), 0.02, device="cuda")

    def write(src, dst):
        if writer == "norm":
            fb.moe_ffn_norm_residual(src, w_pre=scale, normed=dst)
        else:
            fb.moe_ffn_add_adapters(src, src, ids[: src.shape[0]], a, b, out=dst)

    def step(i, between=lambda: None):
        write(gates[i], gate)
        between()
        write(sources[i], shared)
        between()
        return layer(shared, gate).clone()

    want = [step(i, torch.cuda.synchronize) for i in range(n)]
    assert not torch.equal(want[0], want[1])
    for _ in range(5):
        got = [step(i) for i in range(n)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    # the gate last; then in a graph, where nothing but the kernels lies between
    outs = [torch.zeros_like(want[0]) for _ in range(n)]
    write(sources[0], shared)
    torch.cuda.synchronize()
    want = []
    for i in range(n):
        write(gates[i], gate)
        torch.cuda.synchronize()
        want.append(layer(shared, gate).clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            write(gates[i], gate)
            layer(shared, gate)
            outs[i].copy_(layer.out)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs, want))

"""The attention half's operators together, as examples/attention_block.py runs them, in front of the expert half of
examples/serving_block.py, against the formulas in 64 bits."""

import importlib.util
import os

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def mod():
    return example("attention_block")


def dense(w, K, group=32):
    codes = w[:, :K // 2]
    q = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double() - 8
    return q * w[:, K // 2:].contiguous().view(torch.float16).double().repeat_interleave(group, 1)


class Reference:
    """The half block in 64 bits, every sequence's keys and values as lists of tokens."""

    def __init__(self, block, count):
        self.b = block
        self.qkv, self.out = dense(block.qkv_w, block.H), dense(block.out_w, block.Q_HEADS * block.D)
        self.k, self.v = [[] for _ in range(count)], [[] for _ in range(count)]

    def turned(self, x, pos):
        half = self.b.D // 2
        ang = pos * self.b.inv_freq.double()
        a, c = x[..., :half], x[..., half:]
        return torch.cat((a * ang.cos() - c * ang.sin(), a * ang.sin() + c * ang.cos()), -1)

    def __call__(self, residual, normed, positions, new, sees=None):
        b, bf = self.b, lambda v: v.to(torch.bfloat16).double()  # noqa: E731  what the tensors between the calls hold
        rows = bf(normed.double() @ self.qkv.T).view(len(positions), -1, b.D)
        out, t = torch.zeros(len(positions), b.Q_HEADS * b.D, dtype=torch.float64, device="cuda"), 0
        for s, n in enumerate(new):
            before = len(self.k[s])
            for j in range(n):
                row = rows[t + j]
                self.k[s].append(bf(self.turned(row[b.Q_HEADS:b.Q_HEADS + b.KV_HEADS], positions[t + j])))
                self.v[s].append(row[b.Q_HEADS + b.KV_HEADS:])
            if n:
                keys, values = torch.stack(self.k[s]), torch.stack(self.v[s])
            for j in range(n):
                q = bf(self.turned(rows[t + j, :b.Q_HEADS], positions[t + j])).view(b.KV_HEADS, -1, b.D)
                score = torch.einsum("kgd,ikd->kgi", q, keys) * b.D**-0.5
                hidden = [before + i for i in range(n) if not (sees[t + j] >> i & 1 if sees else i <= j)]
                score[..., hidden] = -float("inf")
                out[t + j] = torch.einsum("kgi,ikd->kgd", torch.softmax(score, -1), values).flatten()
            t += n
        r = residual.double() + bf(out) @ self.out.T
        return r, r / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-6) * b.pre_w.double()


SEES = [0b1, 0b11, 0b101, 0b1011, 0b10101]


def test_prompts_tokens_and_trees(mod):
    block = mod.AttentionBlock(5)
    seqs, ref = mod.Sequences(block, 3), Reference(block, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    steps = [([17, 1, 40], list(range(17)) + [0] + list(range(40)), None), ([1, 1, 1], [17, 1, 40], None),
             ([5, 5, 5], [p + d for p in (18, 2, 41) for d in (0, 1, 1, 2, 2)], SEES * 3)]
    for new, positions, sees in steps:
        T = sum(new)
        residual = torch.randn(T, block.H, generator=g, device="cuda")
        _, normed = fb.moe_ffn_norm_residual(residual, w_pre=block.pre_w)
        r0 = residual.clone()
        want_r, want_n = ref(r0, normed.clone(), positions, new, sees)
        mask = None if sees is None else torch.tensor(sees, dtype=torch.int32, device="cuda")[:, None]
        block(residual, normed, torch.tensor(positions, dtype=torch.int32, device="cuda"), *seqs.append(new), mask)
        torch.cuda.synchronize()
        # rows, keys, queries and outputs are held in bf16 between the calls.  The reference rounds them too, but what
        # lies next to a border goes the other way: a whole step, 2^-7 relative, of some values.  A row of the last
        # product adds 4096 of them with random signs: 2^-7 of its rms at most, four such roundings, six standard
        # deviations
        bound = 4 * 6 * 2.0**-7 * float((want_r - r0.double()).square().mean().sqrt())
        assert float((residual.double() - want_r).abs().max()) <= bound
        assert float((normed.double() - want_n).abs().max()) <= 2 * bound + 2.0**-8 * float(want_n.abs().max())
        # what the caches hold of every sequence
        for s in range(3):
            n = len(ref.k[s])
            at = [int(seqs.table[s, i // block.PAGE]) * block.PAGE + i % block.PAGE for i in range(n)]
            for cache, want in ((block.k_cache, ref.k[s]), (block.v_cache, ref.v[s])):
                got, want = cache.flatten(0, 1)[at].double(), torch.stack(want)
                # 2048 products in fp32, then a step of bf16 for each of two roundings
                assert float((got - want).abs().max()) <= 2 * 2.0**-7 * float(want.abs().max())


def test_a_whole_block_in_a_graph(mod):
    """Attention half, then expert half, eight sequences' next tokens: the same bits replayed as called."""
    block, experts = mod.AttentionBlock(6), example("serving_block").ServingBlock(7)
    seqs = mod.Sequences(block, 8)
    g = torch.Generator(device="cuda").manual_seed(2)

    def inputs(T):
        residual = torch.randn(T, block.H, generator=g, device="cuda")
        return residual, fb.moe_ffn_norm_residual(residual, w_pre=block.pre_w)[1]

    adapters = torch.arange(-1, 7, dtype=torch.int32, device="cuda")
    residual, normed = inputs(8 * 21)
    block(residual, normed, torch.arange(21, dtype=torch.int32, device="cuda").repeat(8), *seqs.append([21] * 8))
    residual, normed = inputs(8)
    positions, where = torch.full((8,), 21, dtype=torch.int32, device="cuda"), seqs.append([1] * 8)
    r0, n0 = residual.clone(), normed.clone()

    def step():
        block(residual, normed, positions, *where)
        experts(residual, normed, adapters)

    step()
    want = residual.clone(), normed.clone()
    assert bool(want[0].isfinite().all()) and not torch.equal(want[0], r0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        residual.copy_(r0)
        normed.copy_(n0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(residual, want[0]) and torch.equal(normed, want[1])
    assert experts.kept[8]["layer"].status() == 0


def test_the_example_runs(mod):
    mod.main()

"""moe_ffn_execute_routed: the layer for a routing that the caller brings, against the oracle's expert FFN in 64 bits.

Bars as the layer's own parity tests (1e-2 rms + 1e-5, int8 1e-4 rms), and a tighter one where the weights enter the
products exactly (bf16, and 4-bit on the decode path): sums of up to H + I fp32 products, 2e-5 of the largest output.
"""

import numpy as np
import pytest

import datagen
import fusion_backend_gb300 as fb
import oracle
from datagen import ACT_BF16, ACT_F32, WFMT_BF16, WFMT_I8, WFMT_Q4B32, Shapes

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


class Case:
    def __init__(self, s, wfmt, act=ACT_BF16, seed=5):
        self.s, self.wfmt, self.act = s, wfmt, act
        self.layer = datagen.make_layer(seed, s, wfmt)
        self.x = np.stack([datagen.token_x(seed, t, s.H, act) for t in range(s.T)])
        self.x64 = (self.x if act == ACT_F32 else datagen.bf16_to_f32(self.x)).astype(np.float64)
        self.rng = np.random.default_rng(seed)
        self.cache = {}
        dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.d_x = dev(self.x.view(np.int16) if act == ACT_BF16 else self.x)
        self.d_e, self.d_s = dev(self.layer.expert_w), dev(self.layer.shexp_w)
        self.d_g = dev(self.layer.shexp_gate_w.view(np.int16))
        self.m = fb.MoeFFN(s, act, wfmt)
        self.m.workspace.fill_(0x7F)  # whatever an earlier user left

    def routing(self, dropped=0.0, distinct=True):
        s = self.s
        if distinct:
            ids = np.stack([self.rng.permutation(s.E)[: s.top_k] for _ in range(s.T)])
        else:
            ids = self.rng.integers(0, s.E, (s.T, s.top_k))
        ids[self.rng.random((s.T, s.top_k)) < dropped] = -1
        return ids.astype(np.int32), self.rng.random((s.T, s.top_k)).astype(np.float32)

    def ffn(self, e, t):
        if (e, t) not in self.cache:
            s = self.s
            inter = s.Is if e < 0 else s.I
            n = datagen.expert_bytes(self.wfmt, s.H, inter)
            block = self.layer.shexp_w if e < 0 else self.layer.expert_w[e * n:(e + 1) * n]
            self.cache[e, t] = oracle.swiglu_ffn(block, self.wfmt, s.H, inter, self.x64[t])
        return self.cache[e, t]

    def want(self, ids, w, shared, gated):
        out = np.zeros((self.s.T, self.s.H))
        g = datagen.bf16_to_f32(self.layer.shexp_gate_w).astype(np.float64)
        for t in range(self.s.T):
            for j in range(self.s.top_k):
                if 0 <= ids[t, j] < self.s.E:
                    out[t] += float(w[t, j]) * self.ffn(int(ids[t, j]), t)
            if shared:
                out[t] += (sigmoid(self.x64[t] @ g) if gated else 1.0) * self.ffn(-1, t)
        return out

    def run(self, ids, w, shared=True, gated=True, **kw):
        out = self.m.routed(self.d_x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), self.d_e,
                            self.d_s if shared else None, self.d_g if gated else None, **kw)
        torch.cuda.synchronize()
        assert self.m.status() == 0
        return out.cpu().numpy()

    def check(self, ids, w, shared=True, gated=True):
        want = self.want(ids, w, shared, gated)
        got = self.run(ids, w, shared, gated)
        rms = float(np.sqrt(np.mean(want * want)))
        err = float(np.abs(got - want).max())
        exact = self.wfmt == WFMT_BF16 or (self.wfmt == WFMT_Q4B32 and self.s.T <= 8)
        bar = 2e-5 * np.abs(want).max() if exact else 1e-4 * rms if self.wfmt == WFMT_I8 else 1e-2 * rms + 1e-5
        assert err <= bar, (err, bar, rms)
        counts, offsets, perm, active = self.m.routing()
        keep = [sorted({int(e) for e in row if 0 <= e < self.s.E}) for row in ids]
        want_counts = np.bincount([e for row in keep for e in row], minlength=self.s.E)
        np.testing.assert_array_equal(counts, want_counts)
        np.testing.assert_array_equal(offsets, np.concatenate([[0], np.cumsum(want_counts)]))
        np.testing.assert_array_equal(active, np.nonzero(want_counts)[0])
        first = {}
        for i, e in enumerate(ids.reshape(-1)):
            if 0 <= e < self.s.E:
                first.setdefault((int(e), i // self.s.top_k), i)
        np.testing.assert_array_equal(perm[: offsets[-1]], [first[k] for k in sorted(first)])
        return got


SHAPES = [
    (Shapes(1, 2048, 16, 4, 64, 96), WFMT_BF16, ACT_BF16),
    (Shapes(2, 2048, 16, 4, 60, 40), WFMT_Q4B32, ACT_BF16),
    (Shapes(4, 2048, 16, 8, 64, 32), WFMT_BF16, ACT_BF16),
    (Shapes(7, 2048, 40, 3, 40, 64), WFMT_Q4B32, ACT_BF16),
    (Shapes(1, 2048, 16, 4, 64, 40), WFMT_Q4B32, ACT_BF16),
    (Shapes(1, 2048, 16, 4, 64, 40), WFMT_I8, ACT_BF16),
    (Shapes(8, 2048, 16, 2, 48, 40), WFMT_I8, ACT_BF16),
    (Shapes(3, 264, 5, 3, 136, 72), WFMT_BF16, ACT_F32),
    (Shapes(1, 776, 33, 32, 24, 48), WFMT_BF16, ACT_BF16),
    (Shapes(5, 2304, 8, 2, 64, 64), WFMT_BF16, ACT_BF16),
    (Shapes(2, 512, 8, 2, 64, 64), WFMT_I8, ACT_F32),
    (Shapes(2, 512, 8, 2, 64, 64), WFMT_Q4B32, ACT_F32),
    (Shapes(9, 256, 8, 2, 128, 256), WFMT_BF16, ACT_BF16),
    (Shapes(70, 512, 24, 5, 256, 128), WFMT_BF16, ACT_BF16),
    (Shapes(33, 256, 256, 32, 128, 128), WFMT_BF16, ACT_BF16),
    (Shapes(40, 512, 8, 2, 128, 256), WFMT_Q4B32, ACT_BF16),
]
IDS = [f"T{s.T}-H{s.H}-E{s.E}-k{s.top_k}-w{w}" for s, w, _ in SHAPES]


@pytest.mark.parametrize("s,wfmt,act", SHAPES, ids=IDS)
def test_given_routing(s, wfmt, act):
    c = Case(s, wfmt, act)
    ids, w = c.routing()
    c.check(ids, w)
    c.check(ids, w, gated=False)
    c.check(ids, w, shared=False)
    c.check(*c.routing(dropped=0.5))
    ids, w = c.routing(dropped=0.3)
    ids[ids < 0] = s.E          # past the last expert
    ids[0] = -2**31             # a token with none
    w[0] = np.nan               # whatever its weights
    c.check(ids, w)
    c.check(ids, w, shared=False)


@pytest.mark.parametrize("s,wfmt,act", SHAPES, ids=IDS)
def test_no_choice_at_all(s, wfmt, act):
    c = Case(s, wfmt, act)
    ids, w = c.routing()
    ids[:] = -1
    c.check(ids, w)
    got = c.check(ids, w, shared=False)
    assert not got.any()


@pytest.mark.parametrize("s,wfmt,act", SHAPES, ids=IDS)
def test_repeated_ids_add_their_weights(s, wfmt, act):
    c = Case(s, wfmt, act)
    c.check(*c.routing(distinct=False))
    ids, w = c.routing()
    ids[:] = s.E - 1
    c.check(ids, w, gated=False)


@pytest.mark.parametrize("s,wfmt,act", [SHAPES[i] for i in (0, 2, 4, 5, 8, 13)], ids=[IDS[i] for i in (0, 2, 4, 5, 8, 13)])
def test_repeats_streams_graph_and_the_layer_between(s, wfmt, act):
    c = Case(s, wfmt, act)
    ids, w = c.routing(dropped=0.2)
    got = c.run(ids, w)
    # the layer's own router on the same workspace, before and after
    d_r = torch.from_numpy(c.layer.router_w.view(np.int16).copy()).cuda()
    own = c.m(c.d_x, d_r, c.d_e, c.d_s, c.d_g).cpu().numpy()
    for _ in range(3):
        assert c.run(ids, w).tobytes() == got.tobytes()
    assert c.m(c.d_x, d_r, c.d_e, c.d_s, c.d_g).cpu().numpy().tobytes() == own.tobytes()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert c.run(ids, w, stream=side).tobytes() == got.tobytes()
    d_ids, d_w = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    out = torch.zeros((s.T, s.H), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.m.routed(c.d_x, d_ids, d_w, c.d_e, c.d_s, c.d_g, out=out)
        c.m.routed(c.d_x, d_ids, d_w, c.d_e, c.d_s, c.d_g, out=out)
    ids2, w2 = c.routing()
    d_ids.copy_(torch.from_numpy(ids2))
    d_w.copy_(torch.from_numpy(w2))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert out.cpu().numpy().tobytes() == c.run(ids2, w2).tobytes()


@pytest.mark.parametrize("i", [0, 3, 13])
def test_the_layers_own_routing_given_back(i):
    """The ids and weights of the layer's router, given back, give the layer's result."""
    s, wfmt, act = SHAPES[i]
    c = Case(s, wfmt, act)
    ids = torch.empty((s.T, s.top_k), dtype=torch.int32, device="cuda")
    w = torch.empty((s.T, s.top_k), device="cuda")
    d_r = torch.from_numpy(c.layer.router_w.view(np.int16).copy()).cuda()
    own = c.m(c.d_x, d_r, c.d_e, c.d_s, c.d_g, topk_ids=ids, topk_w=w)
    got = c.m.routed(c.d_x, ids, w, c.d_e, c.d_s, c.d_g)
    torch.cuda.synchronize()
    assert torch.equal(own, got)


def test_out_may_be_x():
    s = Shapes(3, 264, 5, 3, 136, 72)
    c = Case(s, WFMT_BF16, ACT_F32)
    ids, w = c.routing()
    want = c.run(ids, w)
    d_ids, d_w = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    x = c.d_x.clone()
    c.m.routed(x, d_ids, d_w, c.d_e, c.d_s, c.d_g, out=x)
    torch.cuda.synchronize()
    assert x.cpu().numpy().tobytes() == want.tobytes()

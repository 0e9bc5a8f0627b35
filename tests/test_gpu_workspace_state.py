"""The decode kernel's grid-wide barriers on a workspace whose words another user has written into between calls, in
part or as a whole: results as on a fresh one."""

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# byte ranges of the workspace's first 4 KB: control words, then the synchronisation words (256: epoch, 264: their
# complement, 272: the two release words, 288: four arrival counters, 384: the blocks' flags)
RANGES = {"header": (0, 320), "epoch": (256, 272), "epoch and release": (256, 288), "release": (272, 288),
          "counters": (288, 320), "all but flags": (0, 384), "half of the flags": (0, 1000), "flags": (384, 4096)}


class Case:
    def __init__(self, T, H, wfmt, given):
        g = torch.Generator(device="cuda").manual_seed(T + H)
        E, k, I, Is = 16, 4, 64, 40
        bf = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.02).bfloat16()  # noqa: E731
        self.m = fb.MoeFFN(fb.Shapes(T, H, E, k, I, Is), fb.ACT_BF16, wfmt)
        if wfmt == fb.W_BF16:
            rows = lambda n: bf(n, H)  # noqa: E731
        else:  # 4-bit codes and fp16 scales
            def rows(n):
                w = torch.randint(0, 256, (n, H // 2 + H // 16), generator=g, device="cuda", dtype=torch.uint8)
                w[:, H // 2:] = torch.full((n, H // 32), 0.004, device="cuda").half().view(torch.uint8)
                return w
        self.args = (bf(T, H) * 50, bf(E, H), rows(E * 3 * I), rows(3 * Is), bf(H))
        self.ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32) if given else None
        self.w = torch.rand(T, k, generator=g, device="cuda")
        # the call's inputs change between calls: old partial sums are not the new ones
        self.xs = [self.args[0].roll(i, 1).contiguous() for i in range(4)]
        self.x = self.xs[0].clone()
        self.out = torch.zeros(T, H, device="cuda")

    def call(self):
        _, router, expert, shared, gate = self.args
        if self.ids is None:
            self.m(self.x, router, expert, shared, gate, out=self.out)
        else:
            self.m.routed(self.x, self.ids, self.w, expert, shared, gate, out=self.out)

    def run(self, i):
        self.x.copy_(self.xs[i])
        self.out.fill_(float("nan"))
        self.call()
        torch.cuda.synchronize()
        assert self.m.status() == 0
        return self.out.clone()


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T,H,wfmt", [(1, 2048, fb.W_BF16), (1, 512, fb.W_BF16), (2, 512, fb.W_BF16),
                                      (4, 2048, fb.W_Q4B32), (3, 256, fb.W_Q4B32), (8, 2048, fb.W_BF16)])
def test_words_of_another_user(T, H, wfmt, given):
    c = Case(T, H, wfmt, given)
    c.m.workspace.zero_()
    want = [c.run(i) for i in range(4)]
    assert not torch.equal(want[0], want[1])
    for name, (lo, hi) in RANGES.items():
        for fill in (0, 1, 0xFF):
            for start in (0, 0x5A):
                c.m.workspace.fill_(start)
                for i in range(8):  # the same words before every call
                    c.m.workspace[lo:hi] = fill
                    assert torch.equal(c.run(i % 4), want[i % 4]), (name, fill, start, i)
                for i in range(3):  # and none of them: the words as the last call left them
                    assert torch.equal(c.run(i), want[i]), (name, fill, start, i)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T", [1, 2, 8])
def test_words_of_another_user_in_a_graph(T, given):
    c = Case(T, 2048, fb.W_BF16, given)
    c.m.workspace.zero_()
    want = [c.run(i) for i in range(4)]
    for name, (lo, hi) in RANGES.items():
        c.m.workspace.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.m.workspace[lo:hi] = 0
            c.call()
            c.call()
        for i in range(8):
            c.x.copy_(c.xs[i % 4])
            c.out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert c.m.status() == 0 and torch.equal(c.out, want[i % 4]), (name, i)


def test_earlier_words_brought_back():
    """The words of two calls ago, whole or without the counters."""
    for given in (False, True):
        for T in (1, 2):
            c = Case(T, 512, fb.W_BF16, given)
            c.m.workspace.zero_()
            want = [c.run(i) for i in range(4)]
            for lo, hi in ((256, 4096), (256, 272), (256, 288), (288, 320), (256, 320)):
                kept = c.m.workspace[lo:hi].clone()
                for i in range(6):
                    assert torch.equal(c.run(i % 4), want[i % 4])
                    if i % 2:
                        c.m.workspace[lo:hi] = kept
                    assert torch.equal(c.run((i + 1) % 4), want[(i + 1) % 4]), (lo, hi, i)

"""moe_ffn_add_adapters against its formula in 64 bits, with the roundings of the two products counted per element."""

import math

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def reference(y, x, ids, a, b, ranks, scales):
    """Result and error bound in 64 bits.  A product of m terms on the tensor cores keeps at least 23 bits after each
    of its additions (m / 8 steps at most, plus the sum of up to 64 parts); A_a x enters the second product as two
    numbers of the type (bf16: 2^-16 of it is lost at most, fp16 less)."""
    n, R, K = a.shape
    out, bound = y.double().clone(), y.double().abs() * 2.0**-24
    for i in range(n):
        t = torch.nonzero(ids == i)[:, 0]
        r = R if ranks is None else max(0, min(R, int(ranks[i])))
        if t.numel() == 0 or r == 0:
            continue
        s = 1.0 if scales is None else float(scales[i])
        ax, bx = a[i, :r].double(), b[i, :, :r].double()
        v = x[t].double() @ ax.T
        dv = (x[t].double().abs() @ ax.abs().T) * (K / 8 + 72) * 2.0**-23 + v.abs() * 2.0**-16
        d = v @ bx.T
        out[t] += s * d
        mag = v.abs() @ bx.abs().T
        bound[t] += abs(s) * (dv @ bx.abs().T + mag * (r / 8 + 8) * 2.0**-23 + d.abs() * 2.0**-22)
        bound[t] += out[t].abs() * 2.0**-24
    return out, bound


def half_step(v, dtype):
    fi = torch.finfo(dtype)
    return v.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def make(T, K, N, R, n, dtype=BF16, ydtype=F32, seed=0, order="mixed", none=0.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rn(T, K + 8 * pad).to(dtype)[:, :K]
    y = rn(T, N + pad).to(ydtype)[:, :N]
    a, b = (rn(n, R, K) / math.sqrt(K)).to(dtype), (rn(n, N, R) * 0.3).to(dtype)
    ids = torch.randint(0, n, (T,), generator=g, device="cuda")
    if order == "runs":
        ids = ids.sort().values
    if none:
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < none, -1 - ids, ids)
    ranks = torch.randint(0, R + 1, (n,), generator=g, device="cuda").int()
    scales = torch.rand(n, generator=g, device="cuda") * 2 - 0.5
    return y, x, ids.int(), a, b, ranks, scales


def check(y, x, ids, a, b, ranks=None, scales=None, in_place=False):
    want, bound = reference(y, x, ids, a, b, ranks, scales)
    if in_place:
        got = fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, scales)
        assert got is y
    else:
        got = fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, scales, out=torch.empty_like(y))
    torch.cuda.synchronize()
    err = (got.double() - want).abs() - bound - half_step(want.abs() + bound, got.dtype)
    assert float(err.max()) <= 0, float(err.max())
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K,N,R,n", [
    (1, 8, 1, 1, 1), (1, 2048, 2048, 16, 4), (2, 256, 96, 8, 1), (7, 264, 130, 4, 3), (8, 1000, 333, 24, 64),
    (33, 512, 1536, 64, 5), (40, 72, 257, 128, 2), (100, 2048, 64, 32, 100), (1030, 136, 200, 17, 9),
    (300, 64, 48, 100, 1),
])
def test_shapes(T, K, N, R, n, dtype):
    for ydtype in (F32, BF16, F16):
        y, x, ids, a, b, ranks, scales = make(T, K, N, R, n, dtype, ydtype, seed=T + K)
        check(y, x, ids, a, b)
        check(y, x, ids, a, b, ranks, scales)
        check(y, x, ids, a, b, None, scales, in_place=True)


@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("T", [5, 64, 777, 2500])
def test_tokens_without_an_adapter(T, order):
    y, x, ids, a, b, ranks, scales = make(T, 128, 320, 16, 7, seed=T, order=order, none=0.4)
    ids[T // 2] = 7  # one past the pool
    ids[0] = 2**31 - 1
    got = check(y, x, ids, a, b, ranks, scales)
    none = (ids < 0) | (ids >= 7)
    assert torch.equal(got[none], y[none])
    got = check(y, x, torch.full_like(ids, -1), a, b)
    assert torch.equal(got, y)


def test_what_lies_beyond_a_rank_does_not_matter():
    y, x, ids, a, b, _, scales = make(50, 256, 256, 32, 4, seed=2)
    ranks = torch.tensor([0, 3, 16, 50], dtype=torch.int32, device="cuda")  # 50: clamped to 32
    for i, r in enumerate([0, 3, 16]):
        a[i, r:] = math.nan
        b[i, :, r:] = math.inf
    check(y, x, ids, a, b, ranks, scales)
    check(y, x, ids, a, b, -ranks - 1, scales)  # negative: none


@pytest.mark.parametrize("pad", [1, 2, 4])
@pytest.mark.parametrize("ydtype", [F32, BF16])
def test_strides(pad, ydtype):
    y, x, ids, a, b, ranks, scales = make(70, 192, 256, 16, 5, BF16, ydtype, seed=pad, pad=pad)
    check(y, x, ids, a, b, ranks, scales)
    wide = torch.zeros(70, 256 + 3, dtype=ydtype, device="cuda")
    want, bound = reference(y, x, ids, a, b, None, scales)
    fb.moe_ffn_add_adapters(y, x, ids, a, b, None, scales, out=wide[:, 1:257])
    torch.cuda.synchronize()
    assert float(((wide[:, 1:257].double() - want).abs() - bound - half_step(want.abs() + bound, ydtype)).max()) <= 0
    assert float(wide[:, 0].abs().max()) == 0 and float(wide[:, 257:].abs().max()) == 0


def test_large_products_of_fp16_adapters():
    """A_a x far beyond fp16's range."""
    y, x, ids, a, b, _, _ = make(20, 512, 128, 16, 2, F16, seed=4)
    check(y, x * 100, ids, a * 1000, (b * 1e-3).to(F16))


def test_one_adapter_of_many_tokens_and_many_adapters_of_one():
    y, x, ids, a, b, _, scales = make(1100, 64, 64, 8, 1100, seed=6)
    check(y, x, torch.arange(1100, device="cuda", dtype=torch.int32), a, b, None, scales)
    check(y, x, torch.full_like(ids, 1099), a, b, None, scales)


def test_repeats_streams_graph():
    y, x, ids, a, b, ranks, scales = make(3000, 512, 512, 32, 9, seed=7)
    o1 = fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, scales, out=torch.empty_like(y))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, scales, out=torch.empty_like(y), stream=side)
    side.synchronize()
    assert torch.equal(o1, o2)
    o3, ws = torch.zeros_like(y), torch.empty(fb.moe_ffn_adapters_workspace(3000, 512, 512, 32), dtype=torch.uint8,
                                              device="cuda")
    ws.fill_(255)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, scales, out=o3, workspace=ws)
    ids.copy_(ids.flip(0))
    graph.replay()
    o1 = fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, scales, out=torch.empty_like(y))
    torch.cuda.synchronize()
    assert torch.equal(o1, o3)


def test_no_tokens():
    y, x, ids, a, b, _, _ = make(1, 64, 64, 8, 2)
    assert fb.moe_ffn_add_adapters(y[:0], x[:0], ids[:0], a, b).shape == (0, 64)

"""How much of A_a x the second product of moe_ffn_add_adapters keeps, where nothing else rounds: rows of A with one
nonzero element, so that the first product is exact, and rows of B with one, so that the second has one term."""

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def picked(T, R, N, n, dtype, exponents, seed):
    """x of 11 (8) random bits, A_a that picks the elements 2 r and 2 r + 1 of x with powers of two, the second 2^-11
    (2^-8) of the first, and B_a that picks one row of A_a x for every column of y: v_r has up to 22 (16) bits, is exact
    in fp32 and lies about 2^exponents[r]."""
    g = torch.Generator().manual_seed(seed)
    bits = 11 if dtype == F16 else 8
    K = 2 * R + (-2 * R) % 8
    x = torch.zeros(T, K)
    x[:, : 2 * R] = torch.randint(2 ** (bits - 1), 2**bits, (T, 2 * R), generator=g).float()
    a = torch.zeros(n, R, K)
    r = torch.arange(R)
    e = torch.tensor(exponents, dtype=torch.float64)
    a[:, r, 2 * r] = (2.0 ** (e - bits)).float()
    a[:, r, 2 * r + 1] = (2.0 ** (e - 2 * bits)).float()
    pick = torch.randint(0, R, (n, N), generator=g)
    b = torch.zeros(n, N, R).scatter_(2, pick[:, :, None], torch.where(torch.rand(n, N, 1, generator=g) < 0.5, -1.0, 1.0))
    ids = torch.randint(0, n, (T,), generator=g).int()
    xd, ad, bd = x.to(dtype), a.to(dtype), b.to(dtype)
    assert torch.equal(xd.float(), x) and torch.equal(ad.float(), a)
    v = (xd.double()[:, None, : 2 * R] * a.double()[ids.long()][:, :, : 2 * R]).sum(2)
    want = (b.double()[ids.long()] * v[:, None, :]).sum(2)
    return xd.cuda(), ad.cuda(), bd.cuda(), ids.cuda(), want.cuda()


# fp16: A holds 2^(e - 11) and 2^(e - 22), from 2^-24 to 2^15
SPREADS = {F16: {"alike": [0, 0, 0, 0], "near": [6, 4, 2, -2], "far": [12, 5, -1, -2], "farther": [26, 12, 0, -2]},
           BF16: {"alike": [0, 0, 0, 0], "far": [20, 8, -4, -20], "farther": [60, 0, -30, -60]}}


@pytest.mark.parametrize("T", [1, 7, 70, 1030])
@pytest.mark.parametrize("dtype,spread", [(d, s) for d in SPREADS for s in SPREADS[d]])
@pytest.mark.parametrize("R", [4, 20, 128])
def test_bits_of_the_first_product(T, R, dtype, spread):
    exps = [SPREADS[dtype][spread][i % 4] for i in range(R)]
    for n in (1, 9):
        for N in (40, 516, 37):
            x, a, b, ids, want = picked(T, R, N, n, dtype, exps, seed=T + R)
            y = torch.zeros(T, N, device="cuda")
            got = fb.moe_ffn_add_adapters(y, x, ids, a, b, out=torch.empty_like(y))
            torch.cuda.synchronize()
            # 22 bits: off by at most half a step of them
            assert float(((got.double() - want).abs() - want.abs() * 2.0**-22).max()) <= 0
            # y of 16 bits: 16 bits of it, then the rounding of the result
            for yd in (BF16, F16):
                fi = torch.finfo(yd)
                if float(want.abs().max()) >= fi.max / 2:
                    continue
                y = torch.zeros(T, N, device="cuda", dtype=yd)
                got = fb.moe_ffn_add_adapters(y, x, ids, a, b, out=torch.empty_like(y))
                torch.cuda.synchronize()
                bound = want.abs() * 2.0**-16
                bound = bound + (want.abs() + bound) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
                assert float(((got.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("scale", [2.0**-100, 2.0**-60, 1.0, 2.0**60])
def test_bits_at_any_size_of_the_whole(scale):
    """fp16: the scaling by a power of two, taken back through the adapter's scale."""
    x, a, b, ids, want = picked(33, 16, 64, 3, F16, [3, 0, -1, -2] * 4, seed=1)
    y = torch.zeros(33, 64, device="cuda")
    got = fb.moe_ffn_add_adapters(y, x, ids, a, b, scales=torch.full((3,), scale, device="cuda"),
                                  out=torch.empty_like(y))
    torch.cuda.synchronize()
    assert float(((got.double() / scale - want).abs() - want.abs() * 2.0**-22).max()) <= 0


@pytest.mark.parametrize("T,N", [(3, 64), (3, 37), (70, 600)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_finite_beside_infinite(T, N, dtype):
    """An element of A_a x past fp16's range, finite, beside an infinite one: the infinity alone decides."""
    x, a, b = torch.ones(T, 64), torch.zeros(1, 4, 64), torch.zeros(1, N, 4)
    x[:, 1] = 32768.0
    a[0, 0, 0], a[0, 1, 1] = float("inf"), 8.0
    sign = torch.where(torch.arange(N) % 2 == 0, 1.0, -1.0)
    b[0, :, 0], b[0, :, 1] = sign, -sign
    y = torch.zeros(T, N, device="cuda")
    got = fb.moe_ffn_add_adapters(y, x.to(dtype).cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"),
                                  a.to(dtype).cuda(), b.to(dtype).cuda(), out=torch.empty_like(y))
    torch.cuda.synchronize()
    assert torch.equal(got, (sign * float("inf")).cuda().expand(T, N))


@pytest.mark.parametrize("T", [3, 64, 300])
@pytest.mark.parametrize("N", [64, 37, 600])
@pytest.mark.parametrize("ydtype", [F32, BF16, F16])
def test_minus_zero_without_an_adapter(T, N, ydtype):
    """A token without an adapter, or with one of rank 0, keeps y bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(T)
    y = torch.where(torch.rand(T, N, generator=g, device="cuda") < 0.5, -0.0, 0.0).to(ydtype)
    bits = torch.int32 if ydtype == F32 else torch.int16
    x = torch.randn(T, 64, generator=g, device="cuda").to(BF16)
    a, b = torch.randn(3, 8, 64, device="cuda").to(BF16), torch.randn(3, N, 8, device="cuda").to(BF16)
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ids[1::2] = 2
    ranks = torch.tensor([8, 8, 0], dtype=torch.int32, device="cuda")
    for got in (fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks, out=torch.ones_like(y)),
                fb.moe_ffn_add_adapters(y.clone(), x, ids, a, b, ranks)):
        torch.cuda.synchronize()
        assert torch.equal(got.view(bits), y.view(bits))

"""moe_ffn_project against its formula in 64 bits."""

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def half_step(v, dtype):
    fi = torch.finfo(dtype)
    return v.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def weights(gen, N, K, group, pad=0):
    """Rows of random codes and scales, `pad` more bytes behind each (multiples of 16 in all)."""
    need = K // 2 + 2 * (K // group)
    row = (need + 15) // 16 * 16 + pad
    w = torch.randint(0, 256, (N, row), generator=gen, device="cuda", dtype=torch.uint8)
    d = (torch.rand(N, K // group, generator=gen, device="cuda") * 0.02 + 0.001).half()
    w[:, K // 2:need] = d.view(torch.uint8)
    return w


def dense(w, K, group):
    codes = w[:, :K // 2]
    q = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double() - 8
    d = w[:, K // 2:K // 2 + 2 * (K // group)].contiguous().view(F16).double()
    return q * d.repeat_interleave(group, 1)


def check(x, w, group, bias, y):
    K = x.shape[1]
    W = dense(w, K, group)
    want, size = x.double() @ W.T, x.double().abs() @ W.abs().T
    if bias is not None:
        want, size = want + bias.double(), size + bias.double().abs()
    # products are exact; at most K / 8 + 40 additions and scalings follow one another, each off by at most a step of
    # fp32 (a tensor core may cut off) of the sum of magnitudes
    err = size * ((K / 8 + 40) * 2.0**-23)
    d = (y.double() - want).abs() - err - half_step(want.abs() + err, y.dtype)
    assert float(d.max()) <= 0, float(d.max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("T,K,N", [(1, 128, 1), (1, 2048, 640), (2, 384, 17), (7, 640, 33), (8, 4096, 100), (9, 128, 16),
                                   (16, 1152, 257), (17, 256, 48), (33, 2048, 65), (61, 896, 130), (64, 128, 31),
                                   (65, 512, 96), (200, 1024, 70), (1, 8192, 24), (3, 1024, 5001)])
def test_values(T, K, N, xt, yt, group):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + K + N)
    x = torch.randn(T, K, generator=g, device="cuda").to(xt)
    w = weights(g, N, K, group)
    bias = torch.randn(N, generator=g, device="cuda") if N % 2 else None
    y = fb.moe_ffn_project(x, w, group=group, bias=bias, out_dtype=yt)
    assert y.dtype == yt and y.shape == (T, N)
    check(x, w, group, bias, y)


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (64, 64), (160, 32), (192, 64), (65536, 128), (65504, 32)])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_few_and_many_columns(T, K, group):
    g = torch.Generator(device="cuda").manual_seed(K)
    x, w = torch.randn(T, K, generator=g, device="cuda").bfloat16(), weights(g, 37, K, group)
    check(x, w, group, None, fb.moe_ffn_project(x, w, group=group, out_dtype=F32))


def test_tokens_and_rows_to_the_limit():
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w = torch.randn(1024, 256, generator=g, device="cuda").half(), weights(g, 75, 256, 32)
    check(x, w, 32, None, fb.moe_ffn_project(x, w))
    with pytest.raises(fb.MoeFFNError):
        fb.moe_ffn_project(torch.zeros(1025, 256, device="cuda", dtype=BF16), w)
    assert fb.moe_ffn_project(x[:0], w).shape == (0, 75)


def test_strides_and_neighbours():
    """x and y inside wider rows, w with bytes behind its rows: nothing beside y changes, whatever lies there."""
    g = torch.Generator(device="cuda").manual_seed(4)
    T, K, N = 13, 512, 45
    full = torch.full((T, K + 24), float("nan"), device="cuda", dtype=BF16)
    full[:, 8:8 + K] = torch.randn(T, K, generator=g, device="cuda")
    x, w = full[:, 8:8 + K], weights(g, N, K, 32, pad=48)
    out = torch.full((T, N + 3), 7.0, device="cuda", dtype=BF16)
    y = fb.moe_ffn_project(x, w, out=out[:, 1:1 + N])
    check(x, w, 32, None, y)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 1 + N:] == 7).all())
    # rows in another order, taken from a wider matrix of the layer's
    check(x, w[4::3], 32, None, fb.moe_ffn_project(x, w[4::3]))


def test_the_layers_rows():
    """A stored matrix of the layer's 4-bit format, as it lies in the layer's weights."""
    import numpy as np

    import datagen

    s = datagen.Shapes(1, 512, 4, 2, 128, 256)
    layer = datagen.make_layer(3, s, datagen.WFMT_Q4B32)
    w = torch.from_numpy(layer.shexp_w.view(np.uint8).reshape(3 * 256, -1)).cuda()
    x = torch.randn(3, 512, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    check(x, w[:256], 32, None, fb.moe_ffn_project(x, w[:256], out_dtype=F32))


def test_large_offsets():
    """Rows of W behind 4 GB."""
    K, N = 2048, 300
    row = 2**24
    if torch.cuda.mem_get_info()[0] < 12 * 2**30:
        pytest.skip("needs 6 GB")
    big = torch.empty((N, row), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    w = weights(g, N, K, 32)
    big[:, :w.shape[1]] = w
    x = torch.randn(2, K, generator=g, device="cuda").bfloat16()
    got = fb.moe_ffn_project(x, big[:, :w.shape[1]], out_dtype=F32)
    assert torch.equal(got, fb.moe_ffn_project(x, w, out_dtype=F32))


@pytest.mark.parametrize("T", [1, 20])
def test_infinities_stay_in_their_token(T):
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = torch.randn(T + 1, 256, generator=g, device="cuda").bfloat16(), weights(g, 40, 256, 32)
    clean = fb.moe_ffn_project(x, w, out_dtype=F32)
    x[T, 17] = float("inf")
    x[T, 200] = float("nan")
    got = fb.moe_ffn_project(x, w, out_dtype=F32)
    assert torch.equal(got[:T], clean[:T]) and bool(got[T].isnan().all())


@pytest.mark.parametrize("T", [1, 8, 40, 130])
def test_repeats_graphs_and_streams(T):
    g = torch.Generator(device="cuda").manual_seed(6)
    x, w = torch.randn(T, 1024, generator=g, device="cuda").bfloat16(), weights(g, 777, 1024, 64)
    want = fb.moe_ffn_project(x, w, group=64)
    out = torch.empty_like(want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    fb.moe_ffn_project(x, w, group=64, out=out, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.moe_ffn_project(x, w, group=64, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("T,K,N", [(3, 1024, 70001), (8, 2048, 40003), (5, 256, 150001), (3, 4096, 20005), (2, 8192, 50003),
                                   (20, 1024, 30001), (31, 2048, 12007), (12, 2048, 20005), (16, 4096, 20005), (12, 8192, 50003),
                                   (20, 8192, 20005), (100, 1024, 5003), (150, 5120, 3001)])
def test_many_tiles_a_block(T, K, N, xt, group):
    """Every block takes several batches of tiles, every warp more of them than its ring holds."""
    g = torch.Generator(device="cuda").manual_seed(T + N)
    x = torch.randn(T, K, generator=g, device="cuda").to(xt)
    w = weights(g, N, K, group)
    bias = torch.randn(N, generator=g, device="cuda")
    y = fb.moe_ffn_project(x, w, group=group, bias=bias, out_dtype=F32)
    for n in range(0, N, 10007):
        rows = slice(n, n + 10007)
        check(x, w[rows], group, bias[rows], y[:, rows])
    assert torch.equal(fb.moe_ffn_project(x, w, group=group, bias=bias, out_dtype=F32), y)

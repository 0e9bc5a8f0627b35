"""moe_ffn_norm_residual against its formula in 64 bits, with the roundings of an fp32 evaluation counted per element."""

import math

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0**-24  # half a step of fp32, relative


def reference(res, y, post_norm, w_post, gate, sigmoid, alpha, beta, w_pre, w_offset, eps):
    """(r', bound on its fp32 error, normed, bound on its fp32 error) in 64 bits."""
    H = res.shape[1]
    # a sum of H squares in a tree over 32 lanes or more: H / 32 + 10 roundings; its share of an inverse square root
    # is half of that; mean, eps, root, quotient and product: 6 more
    red = (H / 32 + 10) / 2 * U + 6 * U
    weight = lambda w: torch.ones(H, dtype=torch.float64, device=res.device) if w is None else w.double() + w_offset  # noqa: E731
    r = alpha * res.double()
    dr = r.abs() * U
    if y is not None:
        z = y.double()
        dz = torch.zeros_like(z)
        if post_norm:
            z = z / torch.sqrt((z * z).mean(1, keepdim=True) + eps) * weight(w_post)
            dz = z.abs() * (red + 3 * U)
        if gate is not None:
            g = gate.double()
            a = torch.sigmoid(g) if sigmoid else g
            dz = dz * a.abs() + (z * a).abs() * 8 * U
            z = z * a
        r = r + beta * z
        dr = dr + abs(beta) * dz + (beta * z).abs() * 2 * U + r.abs() * U
    rms = torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    n = r / rms * weight(w_pre)
    # the root moves with r' by at most the rms of its errors over rms
    move = torch.sqrt((dr * dr).mean(1, keepdim=True)) / rms
    dn = dr / rms * weight(w_pre).abs() + n.abs() * (move + red + 4 * U)
    return r, dr, n, dn


def half_step(v, dtype):
    """Half a step of dtype at v (subnormals included)."""
    fi = torch.finfo(dtype)
    return v.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def check(res, y=None, post_norm=False, w_post=None, gate=None, sigmoid=False, alpha=1.0, beta=1.0, w_pre=None,
          w_offset=0.0, eps=1e-6, norm_dtype=BF16, in_place=False):
    want_r, dr, want_n, dn = reference(res, y, post_norm, w_post, gate, sigmoid, alpha, beta, w_pre, w_offset, eps)
    target = res.clone() if in_place else None
    out, n = fb.moe_ffn_norm_residual(target if in_place else res, y, post_norm, w_post, gate,
                                      fb.GATE_SIGMOID if sigmoid else fb.GATE_LINEAR, alpha, beta, w_pre, w_offset,
                                      eps, res_out=None if in_place else torch.empty_like(res), norm_dtype=norm_dtype)
    torch.cuda.synchronize()
    assert out.dtype == res.dtype and n.dtype == norm_dtype
    er = (out.double() - want_r).abs() - dr - half_step(want_r.abs() + dr, res.dtype)
    en = (n.double() - want_n).abs() - dn - half_step(want_n.abs() + dn, norm_dtype)
    assert float(er.max()) <= 0 and float(en.max()) <= 0, (float(er.max()), float(en.max()))
    return out, n


def rand(gen, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def make_gate(gen, kind, T, H, dtype):
    return {"none": None, "channel": lambda: rand(gen, H, dtype=dtype), "token": lambda: rand(gen, T, 1, dtype=dtype),
            "full": lambda: rand(gen, T, H, dtype=dtype)}[kind] and {
        "channel": lambda: rand(gen, H, dtype=dtype), "token": lambda: rand(gen, T, 1, dtype=dtype),
        "full": lambda: rand(gen, T, H, dtype=dtype)}[kind]()


@pytest.mark.parametrize("T,H", [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 100), (65, 1024), (4, 2883), (9, 4096),
                                 (3, 5000), (2, 8192), (2, 16391), (1, 32768), (513, 24)])
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
def test_shapes_and_gates(T, H, kind):
    gen = torch.Generator(device="cuda").manual_seed(T * H)
    for i, (yd, rd, nd) in enumerate([(F32, F32, BF16), (BF16, BF16, BF16), (F16, F32, F16), (BF16, F16, F32)]):
        gate = make_gate(gen, kind, T, H, F32 if i % 2 == 0 else yd)
        check(rand(gen, T, H, dtype=rd), rand(gen, T, H, dtype=yd), post_norm=i != 1,
              w_post=rand(gen, H, dtype=F32 if i else BF16) if i != 2 else None, gate=gate, sigmoid=i >= 2, alpha=0.75,
              beta=1.25, w_pre=rand(gen, H, dtype=BF16 if i else F32) if i != 3 else None, w_offset=1.0 if i else 0.0,
              norm_dtype=nd)


@pytest.mark.parametrize("H", [8, 130, 2048, 9001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_alone_and_in_place(H, dtype):
    gen = torch.Generator(device="cuda").manual_seed(H)
    res = rand(gen, 6, H, dtype=dtype)
    kept = res.clone()
    out, _ = fb.moe_ffn_norm_residual(res, norm_dtype=F32)
    assert out is res and torch.equal(res, kept)  # nothing but the norm
    check(res, w_pre=rand(gen, H), norm_dtype=F32)
    check(res, alpha=0.5, w_pre=rand(gen, H), norm_dtype=BF16)
    check(res, rand(gen, 6, H, dtype=BF16), post_norm=True, gate=rand(gen, H), in_place=True)


@pytest.mark.parametrize("pad", [1, 3, 8, 13])
@pytest.mark.parametrize("H", [256, 2883])
def test_strides(H, pad):
    gen = torch.Generator(device="cuda").manual_seed(pad)
    T = 37
    wide = lambda dtype: rand(gen, T, H + pad, dtype=dtype)  # noqa: E731
    for dt in (F32, BF16):
        res, y, gate = wide(dt)[:, :H], wide(dt)[:, pad:], wide(dt)[:, :H]
        want_r, dr, want_n, dn = reference(res, y, True, None, gate, True, 0.9, 0.5, None, 0.0, 1e-6)
        ro, no = wide(dt), wide(BF16)
        kr, kn = ro.clone(), no.clone()
        fb.moe_ffn_norm_residual(res, y, True, None, gate, fb.GATE_SIGMOID, 0.9, 0.5, res_out=ro[:, 1:1 + H],
                                 normed=no[:, :H])
        torch.cuda.synchronize()
        assert float(((ro[:, 1:1 + H].double() - want_r).abs() - dr - half_step(want_r.abs() + dr, dt)).max()) <= 0
        assert float(((no[:, :H].double() - want_n).abs() - dn - half_step(want_n.abs() + dn, BF16)).max()) <= 0
        # the columns between the rows stay as they were
        assert torch.equal(ro[:, :1], kr[:, :1]) and torch.equal(ro[:, 1 + H:], kr[:, 1 + H:])
        assert torch.equal(no[:, H:], kn[:, H:])


def test_normed_over_y():
    gen = torch.Generator(device="cuda").manual_seed(3)
    res, y = rand(gen, 11, 2048), rand(gen, 11, 2048, dtype=BF16)
    want = fb.moe_ffn_norm_residual(res.clone(), y, True)[1]
    y2 = y.clone()
    assert torch.equal(fb.moe_ffn_norm_residual(res.clone(), y2, True, normed=y2)[1], want)


def test_zero_rows_and_large_values():
    res = torch.zeros(3, 512, device="cuda")
    res[1] = 1e15
    res[2] = 1e-18
    y = torch.zeros(3, 512, device="cuda")
    y[1] = -1e15
    y[2, 7] = 3e-20
    check(res, y, post_norm=True, norm_dtype=F32)
    check(res, y, post_norm=True, eps=0.25, norm_dtype=BF16)
    out, n = fb.moe_ffn_norm_residual(res[:1].clone(), y[:1], post_norm=True, norm_dtype=F32)
    assert float(out.abs().max()) == 0 and float(n.abs().max()) == 0


def test_nan_stays_in_its_row():
    res = torch.ones(4, 300, device="cuda")
    res[2, 5] = math.nan
    _, n = fb.moe_ffn_norm_residual(res, norm_dtype=F32)
    torch.cuda.synchronize()
    assert bool(torch.isnan(n[2]).all()) and not bool(torch.isnan(n[[0, 1, 3]]).any())


def test_repeats_streams_graph():
    gen = torch.Generator(device="cuda").manual_seed(8)
    res, y, g = rand(gen, 700, 2048), rand(gen, 700, 2048), rand(gen, 2048)
    r1, n1 = fb.moe_ffn_norm_residual(res, y, True, gate=g, res_out=torch.empty_like(res))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2 = torch.empty_like(res)
    r2, n2 = fb.moe_ffn_norm_residual(res, y, True, gate=g, res_out=r2, stream=side)
    side.synchronize()
    assert torch.equal(r1, r2) and torch.equal(n1, n2)
    r3, n3 = torch.zeros_like(res), torch.zeros_like(n1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.moe_ffn_norm_residual(res, y, True, gate=g, res_out=r3, normed=n3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r1, r3) and torch.equal(n1, n3)


def test_no_tokens():
    r, n = fb.moe_ffn_norm_residual(torch.zeros(0, 64, device="cuda"))
    assert r.shape == n.shape == (0, 64)


@pytest.mark.parametrize("H", [516, 1024, 2048, 2052, 4096, 6000, 8192])
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
def test_many_rows(H, kind):
    """More rows than the GPU holds at once, in every combination of element sizes."""
    T = 1300 if H < 4000 else 700
    gen = torch.Generator(device="cuda").manual_seed(H)
    for i, (yd, rd, nd) in enumerate([(F32, F32, BF16), (BF16, F32, F32), (F16, BF16, F16), (F32, BF16, F32)]):
        gate = make_gate(gen, kind, T, H, yd)
        check(rand(gen, T, H, dtype=rd), rand(gen, T, H, dtype=yd), post_norm=i != 2, w_post=rand(gen, H) if i else None,
              gate=gate, sigmoid=i % 2 == 1, alpha=0.75, beta=1.25, w_pre=rand(gen, H, dtype=BF16) if i != 1 else None,
              w_offset=1.0, norm_dtype=nd, in_place=i == 3)


@pytest.mark.parametrize("H", [520, 2048, 5000])
def test_many_rows_norm_alone_and_padded(H):
    gen = torch.Generator(device="cuda").manual_seed(H + 1)
    T = 900
    check(rand(gen, T, H), w_pre=rand(gen, H), norm_dtype=F32)
    check(rand(gen, T, H, dtype=BF16), alpha=0.5, w_pre=rand(gen, H))
    # rows of a wider matrix; outputs left out in turn
    res, y = rand(gen, T, H + 12)[:, :H], rand(gen, T, H + 8, dtype=BF16)[:, :H]
    want_r, dr, want_n, dn = reference(res, y, True, None, None, False, 1.0, 1.0, None, 0.0, 1e-6)
    out, n = fb.moe_ffn_norm_residual(res, y, True, res_out=torch.empty(T, H, device="cuda"), norm_dtype=F32)
    assert float(((out.double() - want_r).abs() - dr - half_step(want_r.abs() + dr, F32)).max()) <= 0
    assert float(((n.double() - want_n).abs() - dn - half_step(want_n.abs() + dn, F32)).max()) <= 0
    _, only = fb.moe_ffn_norm_residual(res, norm_dtype=F32)
    want = reference(res, None, False, None, None, False, 1.0, 1.0, None, 0.0, 1e-6)
    assert float(((only.double() - want[2]).abs() - want[3] - half_step(want[2].abs() + want[3], F32)).max()) <= 0
    # a zero row between others: nothing of theirs may reach it
    res = rand(gen, T, H)
    res[T // 2] = 0
    _, n = fb.moe_ffn_norm_residual(res, norm_dtype=F32)
    assert float(n[T // 2].abs().max()) == 0


def test_residual_alone():
    """No second norm: the C entry with normed left out."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    for T, H in ((3, 100), (700, 2048), (700, 2050)):
        res, y = rand(gen, T, H), rand(gen, T, H)
        want = fb.moe_ffn_norm_residual(res, y, True, res_out=torch.empty_like(res))[0]
        out = torch.zeros_like(res)
        a = fb.NormArgs(T, H, 0, 0, 1, 0, 0, 0, 1, 0, 0, 1.0, 1.0, 0.0, 1e-6, H, H, H, H, H)
        rc = fb.lib().moe_ffn_norm_residual(a, torch.cuda.current_stream().cuda_stream, res.data_ptr(), y.data_ptr(),
                                            None, None, None, out.data_ptr(), None)
        torch.cuda.synchronize()
        assert rc == fb.OK and torch.equal(out, want)


@pytest.mark.parametrize("H", [517, 1026, 2883, 4095])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_rows_of_any_alignment(H, dtype):
    """More rows than four an SM whose starts go through every offset from a four-element boundary."""
    gen = torch.Generator(device="cuda").manual_seed(H)
    T = 640
    wide = lambda pad, dt=dtype: rand(gen, T, H + pad, dtype=dt)  # noqa: E731
    # every tensor at an offset of its own; then one of them in fp32, each in turn, and rows on the boundary
    for odd, pads in ((None, (1, 2, 3, 4, 5)), (0, (3, 1, 1, 2, 7)), (1, (5, 3, 2, 1, 2)), (2, (2, 5, 7, 3, 1)),
                      (3, (1, 1, 1, 1, 1)), (None, tuple([-H % 4] * 5))):
        dts = [F32 if odd == i else dtype for i in range(4)]  # res, y, gate, normed
        res, y, gate = (wide(p, d)[:, p // 2:p // 2 + H] for p, d in zip(pads, dts[:3]))
        w_post, w_pre = rand(gen, H + 1, dtype=BF16)[1:], rand(gen, H)
        want_r, dr, want_n, dn = reference(res, y, True, w_post, gate, True, 0.9, 0.5, w_pre, 1.0, 1e-6)
        ro, no = wide(pads[3], dts[0]), wide(pads[4], dts[3])
        kr, kn = ro.clone(), no.clone()
        fb.moe_ffn_norm_residual(res, y, True, w_post, gate, fb.GATE_SIGMOID, 0.9, 0.5, w_pre, 1.0,
                                 res_out=ro[:, pads[3] - 1:][:, :H] if pads[3] else ro, normed=no[:, :H])
        torch.cuda.synchronize()
        first = max(pads[3] - 1, 0)
        got = ro[:, first:first + H].double()
        assert float(((got - want_r).abs() - dr - half_step(want_r.abs() + dr, dts[0])).max()) <= 0
        assert float(((no[:, :H].double() - want_n).abs() - dn - half_step(want_n.abs() + dn, dts[3])).max()) <= 0
        assert torch.equal(ro[:, :first], kr[:, :first]) and torch.equal(ro[:, first + H:], kr[:, first + H:])
        assert torch.equal(no[:, H:], kn[:, H:])
    # in place, without a norm between the reads and the writes
    check(rand(gen, T, H, dtype=dtype), rand(gen, T, H, dtype=dtype), alpha=0.5, in_place=True)
    check(rand(gen, T, H, dtype=dtype), alpha=0.5, in_place=True, norm_dtype=dtype)


def test_a_row_ends_where_the_neighbour_holds_nan():
    """What lies before, behind and between the rows enters no row."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    for T, H in ((3, 61), (640, 517), (640, 2883)):
        for shift in range(4):
            hold = torch.full((T, H + 7), math.nan, dtype=BF16, device="cuda")
            hold[:, shift + 1:shift + 1 + H] = rand(gen, T, H, dtype=BF16)
            res = hold[:, shift + 1:shift + 1 + H]
            check(res, res.clone(), post_norm=True, gate=res.clone(), w_pre=rand(gen, H))

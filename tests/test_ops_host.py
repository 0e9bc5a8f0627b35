"""Refusals of the operators around the layer, on the host: argument blocks that the library rejects before it touches
a device, and tensors that the binding rejects before it calls the library."""

import ctypes

import pytest

import fusion_backend_gb300 as fb

torch = pytest.importorskip("torch")

P = 4096  # an aligned non-null address that no call here may reach


@pytest.fixture(scope="module")
def lib():
    fb.build()
    return fb.lib()


def route_args(**kw):
    a = fb.RouteArgs(4, 64, 8, fb.SCORE_SIGMOID, 8, 4, fb.GROUP_TOP2, 1, fb.ACT_BF16, 1.0, 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize(
    "change,status",
    [
        (dict(T=-1), fb.ERR_INVALID_ARG),
        (dict(dtype=3), fb.ERR_INVALID_ARG),
        (dict(score=2), fb.ERR_INVALID_ARG),
        (dict(group_score=-1), fb.ERR_INVALID_ARG),
        (dict(scale=float("nan")), fb.ERR_INVALID_ARG),
        (dict(scale=float("inf")), fb.ERR_INVALID_ARG),
        (dict(row_stride=63), fb.ERR_INVALID_ARG),
        (dict(E=0), fb.ERR_UNSUPPORTED),
        (dict(E=1032, row_stride=1032), fb.ERR_UNSUPPORTED),
        (dict(top_k=0), fb.ERR_UNSUPPORTED),
        (dict(top_k=33), fb.ERR_UNSUPPORTED),
        (dict(groups=0), fb.ERR_UNSUPPORTED),
        (dict(groups=7), fb.ERR_UNSUPPORTED),       # not a divisor of E
        (dict(groups=64), fb.ERR_UNSUPPORTED),      # more than 32 groups
        (dict(top_groups=0), fb.ERR_UNSUPPORTED),
        (dict(top_groups=9), fb.ERR_UNSUPPORTED),
        (dict(top_groups=1, top_k=9), fb.ERR_UNSUPPORTED),  # a group of 8 has no 9 experts
    ],
)
def test_route_refuses(lib, change, status):
    assert lib.moe_ffn_route(route_args(**change), None, P, None, P, P) == status


def test_route_refuses_pointers(lib):
    assert lib.moe_ffn_route(None, None, P, None, P, P) == fb.ERR_INVALID_ARG
    for ptrs in ((None, P, P), (P, None, P), (P, P, None)):
        assert lib.moe_ffn_route(route_args(), None, ptrs[0], None, ptrs[1], ptrs[2]) == fb.ERR_INVALID_ARG
    assert lib.moe_ffn_route(route_args(), None, P + 1, None, P, P) == fb.ERR_MISALIGNED
    assert lib.moe_ffn_route(route_args(dtype=fb.ACT_F32), None, P + 2, None, P, P) == fb.ERR_MISALIGNED
    assert lib.moe_ffn_route(route_args(), None, P, P + 2, P, P) == fb.ERR_MISALIGNED
    assert lib.moe_ffn_route(route_args(), None, P, None, P + 2, P) == fb.ERR_MISALIGNED


def norm_args(**kw):
    a = fb.NormArgs(4, 64, 0, 0, 1, 0, 0, 1, 1, fb.GATE_LINEAR, 0, 1.0, 1.0, 0.0, 1e-6, 64, 64, 64, 64, 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize(
    "change,status",
    [
        (dict(T=-1), fb.ERR_INVALID_ARG),
        (dict(y_dtype=3), fb.ERR_INVALID_ARG),
        (dict(res_dtype=-1), fb.ERR_INVALID_ARG),
        (dict(normed_dtype=9), fb.ERR_INVALID_ARG),
        (dict(gate_dtype=4), fb.ERR_INVALID_ARG),
        (dict(w_post_dtype=fb.ACT_F16), fb.ERR_INVALID_ARG),
        (dict(w_pre_dtype=fb.ACT_F16), fb.ERR_INVALID_ARG),
        (dict(gate_layout=3), fb.ERR_INVALID_ARG),
        (dict(eps=-1e-6), fb.ERR_INVALID_ARG),
        (dict(eps=float("nan")), fb.ERR_INVALID_ARG),
        (dict(alpha=float("inf")), fb.ERR_INVALID_ARG),
        (dict(y_stride=63), fb.ERR_INVALID_ARG),
        (dict(res_stride=0), fb.ERR_INVALID_ARG),
        (dict(res_out_stride=1), fb.ERR_INVALID_ARG),
        (dict(normed_stride=-64), fb.ERR_INVALID_ARG),
        (dict(gate_layout=2, gate_stride=63), fb.ERR_INVALID_ARG),
        (dict(gate_layout=1, gate_stride=0), fb.ERR_INVALID_ARG),
        (dict(H=0), fb.ERR_UNSUPPORTED),
        (dict(H=32769), fb.ERR_UNSUPPORTED),
    ],
)
def test_norm_refuses(lib, change, status):
    assert lib.moe_ffn_norm_residual(norm_args(**change), None, P, P, P, P, P, P, P) == status


def test_norm_refuses_pointers(lib):
    f = lib.moe_ffn_norm_residual
    assert f(None, None, P, P, P, P, P, P, P) == fb.ERR_INVALID_ARG
    assert f(norm_args(), None, None, P, P, P, P, P, P) == fb.ERR_INVALID_ARG
    assert f(norm_args(), None, P, P, P, P, P, None, None) == fb.ERR_INVALID_ARG  # nothing to write
    for i in range(7):
        ptrs = [P] * 7
        ptrs[i] += 1
        assert f(norm_args(), None, *ptrs) == fb.ERR_MISALIGNED, i


def adapters_args(**kw):
    a = fb.AdaptersArgs(4, 64, 96, 16, 3, fb.ACT_BF16, fb.ACT_F32, 64, 96, 96)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize(
    "change,status",
    [
        (dict(T=-1), fb.ERR_INVALID_ARG),
        (dict(n_adapters=-1), fb.ERR_INVALID_ARG),
        (dict(x_dtype=fb.ACT_F32), fb.ERR_INVALID_ARG),
        (dict(y_dtype=3), fb.ERR_INVALID_ARG),
        (dict(x_stride=56), fb.ERR_INVALID_ARG),
        (dict(y_stride=95), fb.ERR_INVALID_ARG),
        (dict(out_stride=95), fb.ERR_INVALID_ARG),
        (dict(x_stride=68), fb.ERR_MISALIGNED),
        (dict(R=0), fb.ERR_UNSUPPORTED),
        (dict(R=129), fb.ERR_UNSUPPORTED),
        (dict(K=60), fb.ERR_UNSUPPORTED),
        (dict(K=0), fb.ERR_UNSUPPORTED),
        (dict(N=0), fb.ERR_UNSUPPORTED),
        (dict(T=(1 << 24) + 1), fb.ERR_UNSUPPORTED),
    ],
)
def test_adapters_refuse(lib, change, status):
    ws = ctypes.c_size_t()
    assert lib.moe_ffn_adapters_workspace(adapters_args(**change), ctypes.byref(ws)) == status
    assert lib.moe_ffn_add_adapters(adapters_args(**change), None, P, 1 << 20, P, P, P, P, P, P, P, P) == status


def test_adapters_refuse_pointers_and_workspace(lib):
    f = lib.moe_ffn_add_adapters
    ws = ctypes.c_size_t()
    assert lib.moe_ffn_adapters_workspace(adapters_args(), None) == fb.ERR_INVALID_ARG
    assert lib.moe_ffn_adapters_workspace(adapters_args(), ctypes.byref(ws)) == fb.OK and ws.value % 256 == 0
    assert f(adapters_args(), None, P, ws.value - 1, P, P, P, P, P, P, P, P) == fb.ERR_WORKSPACE
    assert f(adapters_args(), None, None, 1 << 20, P, P, P, P, P, P, P, P) == fb.ERR_INVALID_ARG
    order = (0, 1, 2, 3, 6, 7)  # x, ids, A, B, y, out are required
    for i in order:
        ptrs = [P] * 8
        ptrs[i] = None
        assert f(adapters_args(), None, P, 1 << 20, *ptrs) == fb.ERR_INVALID_ARG, i
    assert f(adapters_args(), None, P + 128, 1 << 20, *[P] * 8) == fb.ERR_MISALIGNED
    for i in range(8):
        ptrs = [P] * 8
        ptrs[i] += 8 if i in (0, 2, 3) else 1
        assert f(adapters_args(), None, P, 1 << 20, *ptrs) == fb.ERR_MISALIGNED, i


def test_no_tokens_is_a_call_that_does_nothing(lib):
    assert lib.moe_ffn_route(route_args(T=0), None, None, None, None, None) == fb.OK
    assert lib.moe_ffn_norm_residual(norm_args(T=0), None, None, None, None, None, None, None, None) == fb.OK
    assert lib.moe_ffn_add_adapters(adapters_args(T=0), None, None, 0, *[None] * 8) == fb.OK


# ---- the binding's own checks (tensors on the CPU: a call that passes every other check stops at the device)


def test_binding_checks_route():
    lg = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fb.moe_ffn_route(lg, 2)
    with pytest.raises(ValueError, match="dtype"):
        fb.moe_ffn_route(lg.double(), 2)
    with pytest.raises(ValueError, match="adjacent"):
        fb.moe_ffn_route(lg.t().contiguous().t(), 2)
    with pytest.raises(ValueError, match="bias"):
        fb.moe_ffn_route(lg, 2, bias=torch.zeros(15))
    with pytest.raises(ValueError, match="ids"):
        fb.moe_ffn_route(lg, 2, ids=torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="weights"):
        fb.moe_ffn_route(lg, 2, weights=torch.zeros(4, 3))


def test_binding_checks_norm():
    r = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fb.moe_ffn_norm_residual(r, r.clone(), gate=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="y: shape"):
        fb.moe_ffn_norm_residual(r, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="gate"):
        fb.moe_ffn_norm_residual(r, r, gate=torch.zeros(15))
    with pytest.raises(ValueError, match="gate"):
        fb.moe_ffn_norm_residual(r, r, gate=torch.zeros(3, 16))
    with pytest.raises(ValueError, match="w_pre"):
        fb.moe_ffn_norm_residual(r, w_pre=torch.zeros(16, dtype=torch.float16))
    with pytest.raises(ValueError, match="res_out"):
        fb.moe_ffn_norm_residual(r, r, res_out=r.bfloat16())
    with pytest.raises(ValueError, match="normed"):
        fb.moe_ffn_norm_residual(r, normed=torch.zeros(4, 16).bfloat16(), norm_dtype=torch.float32)


def test_binding_checks_adapters():
    bf = torch.bfloat16
    x, y, ids = torch.zeros(4, 16, dtype=bf), torch.zeros(4, 24), torch.zeros(4, dtype=torch.int32)
    a, b = torch.zeros(3, 8, 16, dtype=bf), torch.zeros(3, 24, 8, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        fb.moe_ffn_add_adapters(y, x, ids, a, b)
    with pytest.raises(ValueError, match="x: dtype"):
        fb.moe_ffn_add_adapters(y, x.float(), ids, a, b)
    with pytest.raises(ValueError, match="a: "):
        fb.moe_ffn_add_adapters(y, x, ids, a.half(), b)
    with pytest.raises(ValueError, match="b: "):
        fb.moe_ffn_add_adapters(y, x, ids, a, b[:, :, :4])
    with pytest.raises(ValueError, match="adapter_ids"):
        fb.moe_ffn_add_adapters(y, x, ids.long(), a, b)
    with pytest.raises(ValueError, match="ranks"):
        fb.moe_ffn_add_adapters(y, x, ids, a, b, ranks=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="out"):
        fb.moe_ffn_add_adapters(y, x, ids, a, b, out=y.bfloat16())


def test_execute_routed_refuses(lib):
    plan, ws = fb.moe_ffn_prepare(fb.Shapes(2, 256, 8, 2, 128, 128), fb.ACT_BF16, fb.W_BF16)
    f = lib.moe_ffn_execute_routed
    try:
        assert f(None, None, P, ws, P, P, P, P, P, P, P) == fb.ERR_INVALID_ARG
        for i in (0, 2, 3, 4, 5, 8):  # workspace, x, ids, w, expert_w, out are required
            a = [P, ws, P, P, P, P, P, P, P]
            a[i] = None
            assert f(plan, None, *a) == fb.ERR_INVALID_ARG, i
        assert f(plan, None, P, ws - 1, P, P, P, P, P, P, P) == fb.ERR_WORKSPACE
        for i, off in ((0, 128), (2, 8), (3, 2), (4, 2), (5, 8), (6, 8), (7, 8), (8, 8)):
            a = [P, ws, P, P, P, P, P, P, P]
            a[i] += off
            assert f(plan, None, *a) == fb.ERR_MISALIGNED, i
    finally:
        fb.moe_ffn_destroy(plan)


def test_binding_checks_routed():
    m = fb.MoeFFN.__new__(fb.MoeFFN)
    m.plan, m.shapes = None, fb.Shapes(2, 256, 8, 2, 128, 128)
    x, ids, w = torch.zeros(2, 256), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        m.routed(x, ids, w, x)
    with pytest.raises(ValueError, match="ids"):
        m.routed(x, ids.long(), w, x)
    with pytest.raises(ValueError, match="weights"):
        m.routed(x, ids, w[:, :1], x)

"""Refusals of the attention half's operators, on the host: argument blocks that the library rejects before it touches a
device, and tensors that the binding rejects before it calls the library."""

import ctypes

import pytest

import fusion_backend_gb300 as fb

torch = pytest.importorskip("torch")

P = 4096  # an aligned non-null address that no call here may reach
BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    fb.build()
    return fb.lib()


def changed(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def project_args(**kw):
    return changed(fb.ProjectArgs(4, 256, 64, 32, fb.ACT_BF16, fb.ACT_F32, 256, 64, 144), kw)


INVALID, UNSUPPORTED, MISALIGNED = fb.ERR_INVALID_ARG, fb.ERR_UNSUPPORTED, fb.ERR_MISALIGNED


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(x_dtype=fb.ACT_F32), INVALID), (dict(x_dtype=3), INVALID), (dict(y_dtype=-1), INVALID),
    (dict(x_stride=255), INVALID), (dict(y_stride=63), INVALID), (dict(w_stride=128), INVALID), (dict(w_stride=0), INVALID),
    (dict(w_stride=-144), INVALID), (dict(T=1025), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(K=0), UNSUPPORTED), (dict(K=240), UNSUPPORTED), (dict(K=65568), UNSUPPORTED), (dict(K=-32), UNSUPPORTED),
    (dict(group=64, K=288), UNSUPPORTED), (dict(N=0), UNSUPPORTED), (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(w_stride=1 << 40), UNSUPPORTED),
    (dict(x_stride=260), MISALIGNED), (dict(w_stride=152), MISALIGNED)])
def test_project_refuses(lib, change, status):
    assert lib.moe_ffn_project(project_args(**change), None, P, P, P, P) == status


def test_project_refuses_pointers(lib):
    f = lib.moe_ffn_project
    assert f(None, None, P, P, P, P) == INVALID
    for i in (0, 1, 3):
        ptrs = [P] * 4
        ptrs[i] = None
        assert f(project_args(), None, *ptrs) == INVALID, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2)):
        ptrs = [P] * 4
        ptrs[i] += off
        assert f(project_args(), None, *ptrs) == MISALIGNED, i
    assert f(project_args(T=0), None, None, None, None, None) == fb.OK


def append_args(**kw):
    return changed(fb.AppendArgs(4, 8, 2, 64, 64, 0, 1, 1, 1, 16, 10, 1.0, 512, 64, 128, 64, 128, 64, 512, 64,
                                 2048, 128, 64, 2048, 128, 64), kw)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(pages=-1), INVALID), (dict(q_heads=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(x_dtype=3), INVALID), (dict(q_out_dtype=-1), INVALID), (dict(cache_dtype=9), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID)]
    + [({n: 63}, INVALID) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride", "v_head_stride",
                                    "q_out_stride", "q_out_head_stride", "kc_page_stride", "kc_slot_stride",
                                    "kc_head_stride", "vc_page_stride", "vc_slot_stride", "vc_head_stride")]
    + [(dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(kv_heads=0), UNSUPPORTED), (dict(kv_heads=4097), UNSUPPORTED),
       (dict(q_heads=4097), UNSUPPORTED), (dict(D=0), UNSUPPORTED), (dict(D=513), UNSUPPORTED), (dict(rot=-2), UNSUPPORTED),
       (dict(rot=66), UNSUPPORTED), (dict(rot=31), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
       (dict(page_size=1 << 16, pages=1 << 15), UNSUPPORTED)])
def test_append_refuses(lib, change, status):
    assert lib.moe_ffn_append_kv(append_args(**change), None, *[P] * 9) == status


def test_append_refuses_pointers(lib):
    f = lib.moe_ffn_append_kv
    assert f(None, None, *[P] * 9) == INVALID
    for i in range(9):
        ptrs = [P] * 9
        ptrs[i] = None
        assert f(append_args(), None, *ptrs) == INVALID, i
        ptrs[i] = P + 1
        assert f(append_args(), None, *ptrs) == MISALIGNED, i
    assert f(append_args(T=0), None, *[None] * 9) == fb.OK
    assert f(append_args(pages=0), None, *[None] * 9) == fb.OK


def attend_args(**kw):
    return changed(fb.AttendArgs(4, 3, 8, 2, 64, 1, 1, 16, 10, 5, 1, 0.125, 0.0, 512, 64, 512, 64, 2048, 128, 64, 2048, 128,
                                 64, 5, 1), kw)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(pages=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(mask_words=-1), INVALID), (dict(dtype=fb.ACT_F32), INVALID), (dict(dtype=3), INVALID),
    (dict(out_dtype=3), INVALID), (dict(scale=float("nan")), INVALID), (dict(softcap=float("inf")), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(table_stride=4), INVALID), (dict(mask_stride=0), INVALID)]
    + [({n: 56}, INVALID) for n in ("q_stride", "q_head_stride", "out_stride", "out_head_stride", "kc_page_stride",
                                    "kc_slot_stride", "kc_head_stride", "vc_page_stride", "vc_slot_stride", "vc_head_stride")]
    + [({n: 2052}, MISALIGNED) for n in ("kc_page_stride", "kc_slot_stride", "kc_head_stride", "vc_page_stride",
                                         "vc_slot_stride", "vc_head_stride")]
    + [(dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(B=65537), UNSUPPORTED), (dict(kv_heads=0), UNSUPPORTED),
       (dict(q_heads=0), UNSUPPORTED), (dict(q_heads=9), UNSUPPORTED), (dict(q_heads=258), UNSUPPORTED),
       (dict(D=0), UNSUPPORTED), (dict(D=60), UNSUPPORTED), (dict(D=264), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
       (dict(page_size=1 << 20, pages=1 << 11), UNSUPPORTED),
       (dict(page_size=1 << 20, pages=1, max_pages=1025, table_stride=1025), UNSUPPORTED)])
def test_attend_refuses(lib, change, status):
    assert lib.moe_ffn_attend(attend_args(**change), None, P, 1 << 40, *[P] * 9) == status
    n = ctypes.c_size_t()
    assert lib.moe_ffn_attend_workspace(attend_args(**change), ctypes.byref(n)) == status


def test_attend_refuses_pointers(lib):
    f, big = lib.moe_ffn_attend, 1 << 40
    assert f(None, None, P, big, *[P] * 9) == INVALID
    assert f(attend_args(), None, None, big, *[P] * 9) == INVALID
    for i in range(8):
        ptrs = [P] * 9
        ptrs[i] = None
        if i != 6:  # the mask may be missing
            assert f(attend_args(), None, P, big, *ptrs) == INVALID, i
    for i, off in enumerate((1, 8, 8, 2, 2, 2, 2, 1, 2)):
        ptrs = [P] * 9
        ptrs[i] += off
        assert f(attend_args(), None, P, big, *ptrs) == MISALIGNED, i
    assert f(attend_args(), None, P + 128, big, *[P] * 9) == MISALIGNED
    assert f(attend_args(), None, P, 255, *[P] * 9) == fb.ERR_WORKSPACE
    n = ctypes.c_size_t()
    assert lib.moe_ffn_attend_workspace(attend_args(), None) == INVALID
    assert lib.moe_ffn_attend_workspace(attend_args(), ctypes.byref(n)) == fb.OK
    assert f(attend_args(), None, P, n.value - 1, *[P] * 9) == fb.ERR_WORKSPACE
    assert f(attend_args(T=0), None, None, 0, *[None] * 9) == fb.OK
    assert f(attend_args(B=0), None, None, 0, *[None] * 9) == fb.OK


# ---- the binding


class Recorder:
    """Takes any call, keeps its argument block and returns OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(block, *args):
            self.calls.append((name, type(block).from_buffer_copy(block), args))
            return fb.OK

        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(fb, "_lib", r)
    monkeypatch.setattr(fb, "_blocks", {})
    monkeypatch.setattr(fb, "_on_device", lambda first, **tensors: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    return r


z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)  # noqa: E731


def test_project_block(rec):
    x, w = z(3, 80)[:, 8:72], z(5, 64, dtype=torch.uint8)[:, :48]
    out = fb.moe_ffn_project(x, w, out=z(3, 9, dtype=F32)[:, 2:7], stream=1)
    assert out.shape == (3, 5)
    a = rec.calls[0][1]
    assert (a.T, a.K, a.N, a.group, a.x_dtype, a.y_dtype, a.x_stride, a.y_stride, a.w_stride) == (3, 64, 5, 32, 1, 0, 80, 9, 64)


@pytest.mark.parametrize("kw", [
    dict(x=z(3, 64, dtype=F32)), dict(x=z(64)), dict(x=z(3, 128)[:, ::2]), dict(w=z(5, 48, dtype=torch.int8)), dict(w=z(48, dtype=torch.uint8)),
    dict(w=z(5, 35, dtype=torch.uint8)), dict(w=z(5, 96, dtype=torch.uint8)[:, ::2]), dict(group=48), dict(group=128),
    dict(bias=z(4, dtype=F32)), dict(bias=z(5)), dict(out=z(3, 4)), dict(out=z(3, 5, dtype=torch.float64)),
    dict(out=z(3, 5), out_dtype=F32)])
def test_project_refuses_tensors(rec, kw):
    a = dict(x=z(3, 64), w=z(5, 48, dtype=torch.uint8), out=z(3, 5)) | kw
    with pytest.raises(ValueError):
        fb.moe_ffn_project(**a, stream=1)
    assert rec.calls == []


def test_append_block(rec):
    rows = z(3, 10, 16)
    kc, vc = z(7, 2, 4, 16).transpose(1, 2), z(7, 4, 2, 16)
    q_out = fb.moe_ffn_append_kv(rows[:, 6:8], rows[:, 8:], z(3, dtype=I32), z(3, dtype=I32), z(4, dtype=F32), kc, vc,
                                 q=rows[:, :6], interleaved=True, scale=0.5, stream=1)
    assert q_out.data_ptr() == rows.data_ptr()
    a = rec.calls[0][1]
    assert (a.T, a.q_heads, a.kv_heads, a.D, a.rot, a.interleaved, a.page_size, a.pages, a.scale) == (3, 6, 2, 16, 8, 1, 4, 7, 0.5)
    assert (a.q_stride, a.q_head_stride, a.k_stride, a.k_head_stride) == (160, 16, 160, 16)
    assert (a.kc_page_stride, a.kc_slot_stride, a.kc_head_stride) == (128, 16, 64)
    assert (a.vc_page_stride, a.vc_slot_stride, a.vc_head_stride) == (128, 32, 16)


@pytest.mark.parametrize("kw", [
    dict(k=z(3, 2, 16, dtype=F16)), dict(k=z(3, 32)), dict(v=z(3, 2, 8)), dict(v=z(3, 2, 32)[..., ::2]), dict(positions=z(2, dtype=I32)),
    dict(positions=z(3, dtype=torch.int64)), dict(slots=z(3, dtype=torch.int64)), dict(slots=z(6, dtype=I32)[::2]),
    dict(inv_freq=z(9, dtype=F32)), dict(inv_freq=z(4)), dict(inv_freq=z(4, 1, dtype=F32)), dict(k_cache=z(7, 4, 3, 16)),
    dict(k_cache=z(7, 4, 2, 16, dtype=F32)), dict(v_cache=z(6, 4, 2, 16)), dict(k_cache=z(7, 4, 2, 32)[..., ::2]),
    dict(q=z(3, 6, 16, dtype=F32)), dict(q=z(2, 6, 16)), dict(q=z(3, 96)), dict(q_out=z(3, 6, 16)),
    dict(q=z(3, 6, 16), q_out=z(3, 5, 16)), dict(q=z(3, 6, 16), q_out=z(3, 6, 16, dtype=torch.int16))])
def test_append_refuses_tensors(rec, kw):
    a = dict(k=z(3, 2, 16), v=z(3, 2, 16), positions=z(3, dtype=I32), slots=z(3, dtype=I32), inv_freq=z(8, dtype=F32),
             k_cache=z(7, 4, 2, 16), v_cache=z(7, 4, 2, 16)) | kw
    with pytest.raises(ValueError):
        fb.moe_ffn_append_kv(**a, stream=1)
    assert rec.calls == []


def attend_tensors(**kw):
    return dict(q=z(5, 6, 16), k_cache=z(7, 4, 2, 16), v_cache=z(7, 4, 2, 16), page_table=z(3, 2, dtype=I32),
                lens=z(3, dtype=I32), q_start=z(4, dtype=I32), out=z(5, 6, 16), workspace=z(64, dtype=torch.uint8)) | kw


def test_attend_block(rec):
    fb.moe_ffn_attend(**attend_tensors(mask=z(5, 4, dtype=I32)[:, 1:3], softcap=20.0, out=z(5, 8, 20, dtype=F32)[:, 1:7, 2:18]), stream=1)
    a = rec.calls[0][1]
    assert (a.T, a.B, a.q_heads, a.kv_heads, a.D, a.page_size, a.pages, a.max_pages, a.mask_words) == (5, 3, 6, 2, 16, 4, 7, 2, 2)
    assert (a.scale, a.softcap, a.out_stride, a.out_head_stride, a.table_stride, a.mask_stride) == (0.25, 20.0, 160, 20, 2, 4)


@pytest.mark.parametrize("kw", [
    dict(q=z(5, 96)), dict(q=z(5, 6, 16, dtype=F32)), dict(q=z(5, 6, 16, dtype=F16)), dict(q=z(5, 6, 32)[..., ::2]),
    dict(k_cache=z(7, 4, 2, 24)), dict(v_cache=z(7, 4, 3, 16)), dict(v_cache=z(7, 4, 2, 16, dtype=F16)), dict(k_cache=z(7, 8, 16)),
    dict(page_table=z(3, 2, dtype=torch.int64)), dict(page_table=z(6, dtype=I32)), dict(page_table=z(3, 4, dtype=I32)[:, ::2]),
    dict(lens=z(4, dtype=I32)), dict(lens=z(3, dtype=torch.int64)), dict(q_start=z(3, dtype=I32)), dict(q_start=z(4)),
    dict(mask=z(4, 1, dtype=I32)), dict(mask=z(5, 1, dtype=torch.bool)), dict(mask=z(5, dtype=I32)), dict(out=z(5, 6, 8)),
    dict(out=z(5, 6, 16, dtype=torch.int16)), dict(lse=z(5, 6)), dict(lse=z(6, 6, dtype=F32)),
    dict(workspace=z(64, dtype=torch.uint8)[::2])])
def test_attend_refuses_tensors(rec, kw):
    with pytest.raises(ValueError):
        fb.moe_ffn_attend(**attend_tensors(**kw), stream=1)
    assert rec.calls == []


def test_numbers_past_32_bits_are_refused(rec):
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_project(z(1, 64).expand(2**32 + 1, 64), z(1, 48, dtype=torch.uint8), out=z(1, 1).expand(2**32 + 1, 1), stream=1)
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_attend_workspace(2**32 + 1, 1, 8, 2, 64)
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_attend(**attend_tensors(k_cache=z(1, 1, 2, 16).expand(2**32, 1, 2, 16), v_cache=z(1, 1, 2, 16).expand(2**32, 1, 2, 16)), stream=1)
    assert rec.calls == []


def test_another_device_is_refused(rec, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        fb.moe_ffn_project(z(3, 64), z(5, 48, dtype=torch.uint8), out=z(3, 5), stream=1)
    with pytest.raises(ValueError, match="current device"):
        fb.moe_ffn_attend(**attend_tensors(), stream=1)
    with pytest.raises(ValueError, match="current device"):
        fb.moe_ffn_append_kv(z(3, 2, 16), z(3, 2, 16), z(3, dtype=I32), z(3, dtype=I32), None, z(7, 4, 2, 16), z(7, 4, 2, 16), stream=1)
    assert rec.calls == []


def test_a_number_held_in_a_tensor_is_read_on_every_call(rec):
    cap = torch.tensor(10.0)
    a = attend_tensors()
    fb.moe_ffn_attend(**a, softcap=cap, stream=1)
    cap.fill_(30.0)
    fb.moe_ffn_attend(**a, softcap=cap, stream=1)
    assert [c[1].softcap for c in rec.calls] == [10.0, 30.0]


@pytest.mark.parametrize("q_heads,kv_heads,D", [(32, 4, 128), (8, 8, 64), (12, 2, 80), (128, 1, 128), (16, 1, 256)])
def test_a_workspace_serves_smaller_calls(lib, q_heads, kv_heads, D):
    """One that is reported for the largest T and B is large enough for fewer of either, whatever the page size and the
    types: such a call gets as far as the check of its (here misaligned) queries."""
    sizes = (1, 2, 3, 8, 16, 17, 64, 300, 4096)

    def args(T, B, **kw):
        return attend_args(**(dict(T=T, B=B, q_heads=q_heads, kv_heads=kv_heads, D=D) | {n: 4096 for n in (
            "q_stride", "q_head_stride", "out_stride", "out_head_stride", "kc_page_stride", "kc_slot_stride", "kc_head_stride",
            "vc_page_stride", "vc_slot_stride", "vc_head_stride")} | kw))

    def reported(T, B):
        n = ctypes.c_size_t()
        assert lib.moe_ffn_attend_workspace(args(T, B), ctypes.byref(n)) == fb.OK
        return n.value

    for T in sizes:
        for B in sizes:
            have = reported(T, B)
            for t in (s for s in sizes if s <= T):
                for b in (s for s in sizes if s <= B):
                    assert reported(t, b) <= have, (T, B, t, b)
                    for kw in (dict(), dict(page_size=5), dict(out_dtype=fb.ACT_F32), dict(dtype=fb.ACT_F16)):
                        assert lib.moe_ffn_attend(args(t, b, **kw), None, P, have, P + 1, *[P] * 8) == MISALIGNED

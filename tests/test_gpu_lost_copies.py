"""What a kernel leaves when a copy that it waits for never comes: the bounded wait runs out, every result that needed the
copy is NaN, the kernel returns and the next call is right.  The copies themselves all arrive here; the kernels are told
to wait for more bytes than they bring."""

import ctypes
import os
import subprocess

import pytest

import fusion_backend_gb300 as fb
from fusion_backend_gb300 import _build

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """The library's own launches, of lost_copies.cu."""
    out = str(tmp_path_factory.mktemp("lost") / "lost_copies.so")
    lib = fb.build()
    fb.lib()
    subprocess.run([_build.nvcc(), *_build.NVCC_FLAGS, "-I" + _build.CSRC, "-shared", "-o", out,
                    os.path.join(HERE, "lost_copies.cu"), lib, "-Xlinker", "-rpath=" + os.path.dirname(lib)], check=True)
    return ctypes.CDLL(out)


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("T,K,N", [(1, 512, 40), (8, 2048, 33), (12, 512, 17), (29, 1024, 40), (5, 8192, 40), (70, 8192, 40)])
def test_project(launches, T, K, N):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = torch.randint(0, 60, (N, (K // 2 + K // 16 + 15) // 16 * 16), generator=g, device="cuda", dtype=torch.uint8)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    want = fb.moe_ffn_project(x, w, out_dtype=torch.float32)
    for lost in (0, 16, 0):
        y = torch.zeros(T, N, device="cuda")
        torch.cuda.synchronize()
        assert launches.lost_project(T, K, N, 32, sms, lost, ptr(x), ptr(w), ptr(y)) == 0
        torch.cuda.synchronize()
        assert bool(y.isnan().all()) if lost else torch.equal(y, want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend(launches, D):
    """Units of one block and of several, with a sequence that the bounded wait cannot touch: it has no tokens."""
    g = torch.Generator(device="cuda").manual_seed(D)
    lens = [9000, 50, 1, 0, 700]
    pages = sum(-(-n // 16) for n in lens)
    table, at = torch.zeros(5, -(-9000 // 16), dtype=torch.int32), 0
    for b, n in enumerate(lens):
        m = -(-n // 16)
        table[b, :m] = torch.arange(at, at + m)
        at += m
    table = table.cuda()
    k, v = (torch.randn(pages, 16, 2, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(5, 8, D, generator=g, device="cuda").bfloat16()
    lens, starts = torch.tensor(lens, dtype=torch.int32).cuda(), torch.arange(6, dtype=torch.int32).cuda()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(fb.moe_ffn_attend_workspace(5, 5, 8, 2, D), dtype=torch.uint8, device="cuda")
    want, want_lse = torch.zeros_like(q), torch.zeros(5, 8, device="cuda")
    fb.moe_ffn_attend(q, k, v, table, lens, starts, scale=0.125, out=want, lse=want_lse)
    has = lens > 0
    for lost in (0, 16, 0):
        out, lse = torch.full_like(q, 5.0), torch.full((5, 8), 5.0, device="cuda")
        torch.cuda.synchronize()
        assert launches.lost_attend(5, 8, 2, D, 16, pages, table.shape[1], sms, lost, ptr(q), ptr(k), ptr(v), ptr(table),
                                    ptr(lens), ptr(starts), ptr(out), ptr(lse), ptr(ws)) == 0
        torch.cuda.synchronize()
        if lost:
            assert bool(out[has].isnan().all()) and bool(lse[has].isnan().all()) and bool((out[~has] == 0).all())
        else:
            assert torch.equal(out, want) and torch.equal(lse, want_lse)

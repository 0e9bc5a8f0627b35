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

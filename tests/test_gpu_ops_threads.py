"""Calls of different sizes from several host threads, each on a stream of its own: what one call needs of a kernel
that both use is not taken back by the other, and a thread that has made no CUDA call before can make these."""

import ctypes
import shutil
import subprocess
import threading

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HAMMER = r"""
typedef int (*call9_t)(void*, void*, void*, void*, void*, void*, void*, void*, void*);
typedef int (*call10_t)(void*, void*, void*, void*, void*, void*, void*, void*, void*, void*);
extern "C" long hammer(void* f, void** a, long words, long rounds) {
  long bad = 0;
  for (long i = 0; i < rounds; ++i)
    bad += (words == 9 ? ((call9_t)f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8])
                       : ((call10_t)f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9])) != 0;
  return bad;
}
"""


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    """A loop over a C entry of nine or ten words, outside the interpreter and its lock."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("hammer")
    (d / "hammer.cc").write_text(HAMMER)
    subprocess.run([cxx, "-O2", "-shared", "-fPIC", str(d / "hammer.cc"), "-o", str(d / "libhammer.so")], check=True)
    f = ctypes.CDLL(str(d / "libhammer.so")).hammer
    f.restype, f.argtypes = ctypes.c_long, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_long, ctypes.c_long]
    return f


def words(args):
    return (ctypes.c_void_p * len(args))(*[ctypes.addressof(a) if isinstance(a, ctypes.Structure) else a for a in args])


def run_together(hammer, entry, calls, rounds):
    """Every call (its arguments without the stream, which comes second) on a thread and stream of its own,
    `rounds` times; how many of each were refused."""
    start, bad = threading.Barrier(len(calls)), [None] * len(calls)
    streams = [torch.cuda.Stream() for _ in calls]

    def loop(i):
        a = words((calls[i][0], streams[i].cuda_stream, *calls[i][1:]))
        start.wait()
        bad[i] = hammer(ctypes.cast(entry, ctypes.c_void_p), a, len(a), rounds)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_norms_of_different_widths(hammer):
    """Rows of 2048 columns with a gate of every element take six times the shared memory of 516 without one."""
    T = 700
    calls, wants, outs, keep = [], [], [], []
    for H, wide in ((2048, True), (516, False), (2048, True), (516, False)):
        g = torch.Generator(device="cuda").manual_seed(H)
        res, y, gate = (torch.randn(T, H, generator=g, device="cuda") for _ in range(3))
        kw = dict(gate=gate) if wide else {}
        wants.append(fb.moe_ffn_norm_residual(res.clone(), y, True, norm_dtype=torch.float32, **kw)[1])
        out, normed = torch.empty_like(res), torch.empty(T, H, device="cuda")
        outs.append(normed)
        block = fb.NormArgs(T, H, 0, 0, 0, 0, 0, 0, 1, 2, 0, 1.0, 1.0, 0.0, 1e-6, H, H, H, H, H)
        ptr = lambda t: t.data_ptr()  # noqa: E731
        calls.append((block, ptr(res), ptr(y), None, ptr(gate) if wide else None, None, ptr(out),
                      ptr(normed)))
        keep += [res, y, gate, out]
    torch.cuda.synchronize()
    assert run_together(hammer, fb.lib().moe_ffn_norm_residual, calls, 20000) == [0] * 4
    for got, want in zip(outs, wants):
        assert torch.equal(got, want)


def test_batched_layers_of_different_widths(hammer):
    """The router of a batched plan keeps eight rows of x in shared memory: 64 KB at H = 4096, 52 at 3328."""
    calls, wants, outs, keep = [], [], [], []
    for H in (4096, 3328, 4096, 3328):
        T, E, k, I, Is = 16, 4, 2, 128, 128
        g = torch.Generator(device="cuda").manual_seed(H)
        bf = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.02).bfloat16()  # noqa: E731,B023
        x, router, gate, expert, shared = bf(T, H) * 50, bf(E, H), bf(H), bf(E, 3, I, H), bf(3, Is, H)
        m = fb.MoeFFN(fb.Shapes(T, H, E, k, I, Is), fb.ACT_BF16, fb.W_BF16)
        wants.append(m(x, router, expert, shared, gate))
        outs.append(torch.zeros_like(wants[-1]))
        calls.append((m.plan, m.workspace.data_ptr(), m.workspace_bytes,
                      *(t.data_ptr() for t in (x, router, expert, shared, gate, outs[-1]))))
        keep += [x, router, gate, expert, shared, m]
    torch.cuda.synchronize()
    assert run_together(hammer, fb.lib().moe_ffn_execute, calls, 3000) == [0] * 4
    for got, want in zip(outs, wants):
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 16])
def test_layer_on_a_thread_of_its_own(T):
    """The first CUDA calls that a host thread makes are the layer's (tensor maps on both paths)."""
    g = torch.Generator(device="cuda").manual_seed(T)
    bf = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.02).bfloat16()  # noqa: E731
    H, E, k, I, Is = 2048, 8, 2, 128, 128
    x, router, gate, expert, shared = bf(T, H) * 50, bf(E, H), bf(H), bf(E, 3, I, H), bf(3, Is, H)
    m = fb.MoeFFN(fb.Shapes(T, H, E, k, I, Is), fb.ACT_BF16, fb.W_BF16)
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) % E
    w = torch.rand(T, k, generator=g, device="cuda")
    want = m(x, router, expert, shared, gate), m.routed(x, ids, w, expert, shared, gate)
    ptr = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    stream = torch.cuda.Stream()
    for f, args, expect in ((fb.lib().moe_ffn_execute, (x, router, expert, shared, gate), want[0]),
                            (fb.lib().moe_ffn_execute_routed, (x, ids, w, expert, shared, gate), want[1])):
        out, rc = torch.zeros_like(expect), []
        torch.cuda.synchronize()
        a = (m.plan, stream.cuda_stream, m.workspace.data_ptr(), m.workspace_bytes, *ptr(*args, out))
        t = threading.Thread(target=lambda: rc.append(f(*a)))  # noqa: B023
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert rc == [fb.OK] and torch.equal(out, expect)

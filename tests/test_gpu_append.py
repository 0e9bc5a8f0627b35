"""moe_ffn_append_kv against its formula in 64 bits."""

import numpy as np
import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def half_step(v, dtype):
    fi = torch.finfo(dtype)
    return v.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def turned(x, positions, inv_freq, interleaved, scale):
    """(rotated x, bound on its fp32 error) in 64 bits, the angles in numpy's long double."""
    rot = 2 * len(inv_freq)
    ang = positions.cpu().numpy().astype(np.longdouble)[:, None] * inv_freq.cpu().numpy().astype(np.longdouble)
    ang = np.fmod(ang, 2 * np.arccos(np.longdouble(-1))).astype(np.float64)
    cos, sin = (torch.from_numpy(f(ang)).cuda()[:, None] for f in (np.cos, np.sin))
    y = x.double().clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = scale * (a * cos - b * sin), scale * (a * sin + b * cos)
    err = torch.zeros_like(y)
    # sine and cosine: 2 steps of 2^-24 of 1 each and the angle's 2^-33 turns; their scaling, two products and a sum:
    # 4 half steps more
    err[..., ia] = err[..., ib] = abs(scale) * (a.abs() + b.abs()) * 8 * 2.0**-24
    return y, err


def close(got, want, err):
    d = (got.double() - want).abs() - err - half_step(want.abs() + err, got.dtype)
    assert float(d.max()) <= 0, float(d.max())


def caches(gen, pages, page, H, D, dtype, layout):
    def one():
        t = torch.randn((pages, H, page, D) if layout == "head" else (pages, page, H, D), generator=gen, device="cuda")
        t = t.to(dtype)
        return t.transpose(1, 2) if layout == "head" else t

    return one(), one()


def run(T, Hq, Hkv, D, rot, page, xt=BF16, ct=BF16, qt=BF16, interleaved=False, layout="token", scale=1.0, first=0,
        drop=0.0, in_place=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 17 * T + D)
    rows = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(xt)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    pages = (T + page - 1) // page + 2
    kc, vc = caches(g, pages, page, Hkv, D, ct, layout)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if drop:
        slots[torch.rand(T, generator=g, device="cuda") < drop] = -1
    positions = (torch.arange(T, device="cuda") + first).to(torch.int32)
    f = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                  -torch.arange(rot // 2, device="cuda") / max(1, rot // 2)).float()
    wk, ek = turned(k, positions, f, interleaved, scale)
    wq, eq = turned(q, positions, f, interleaved, scale)
    on = slots >= 0
    at = slots[on].long()
    want_k, want_v, err_k = kc.double().clone(), vc.double().clone(), torch.zeros(kc.shape, dtype=torch.float64, device="cuda")
    want_k[at // page, at % page] = wk[on]
    err_k[at // page, at % page] = ek[on]
    want_v[at // page, at % page] = v.double()[on]
    written = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    written[at // page, at % page] = True
    k0, v0 = kc.clone(), vc.clone()
    q_out = None if in_place else torch.full((T, Hq, D), 3.0, device="cuda", dtype=qt)
    q0 = q.clone() if in_place else q_out.clone()
    if Hq:
        got = fb.moe_ffn_append_kv(k, v, positions, slots, f if rot else None, kc, vc, q=q, q_out=q_out,
                                   interleaved=interleaved, scale=scale)
        assert got is (q if in_place else q_out)
        close(got[on], wq[on], eq[on])
        assert torch.equal(got[~on], q0[~on])
    else:
        assert fb.moe_ffn_append_kv(k, v, positions, slots, f if rot else None, kc, vc, interleaved=interleaved,
                                    scale=scale) is None
    close(kc, want_k, err_k)
    close(vc, want_v, 0 * err_k)
    assert torch.equal(kc[~written], k0[~written]) and torch.equal(vc[~written], v0[~written])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page", [
    (1, 32, 4, 128, 128, 16), (8, 32, 4, 128, 128, 16), (3, 4, 4, 64, 32, 1), (5, 8, 1, 256, 64, 64),
    (17, 7, 1, 80, 80, 24), (130, 14, 2, 96, 48, 8), (700, 4, 2, 64, 64, 128), (2, 1, 1, 8, 2, 3), (9, 3, 1, 40, 20, 5),
    (4, 2, 2, 512, 512, 4), (6, 2, 1, 7, 6, 5), (5, 0, 2, 128, 128, 16), (4, 2, 2, 64, 0, 16), (3, 2, 1, 1, 0, 2)])
def test_values(T, Hq, Hkv, D, rot, page, layout, interleaved):
    run(T, Hq, Hkv, D, rot, page, interleaved=interleaved, layout=layout, drop=0.2 if T > 4 else 0.0)


@pytest.mark.parametrize("xt", [F32, BF16, F16])
@pytest.mark.parametrize("ct", [F32, BF16, F16])
@pytest.mark.parametrize("qt", [F32, BF16, F16])
def test_types(xt, ct, qt):
    run(21, 6, 2, 64, 64, 16, xt=xt, ct=ct, qt=qt, scale=1.25)
    run(5, 6, 2, 36, 20, 16, xt=xt, ct=ct, qt=qt, interleaved=True, scale=0.5)


@pytest.mark.parametrize("first", [0, 40000, 1 << 20, (1 << 24) - 3, (1 << 31) - 40, -(1 << 31), -17])
def test_far_positions(first):
    run(32, 4, 2, 128, 128, 16, xt=F32, ct=F32, qt=F32, first=first)
    run(32, 4, 2, 128, 64, 16, xt=F32, ct=F32, qt=F32, first=first, interleaved=True)


@pytest.mark.parametrize("xt", [BF16, F32])
def test_queries_in_place(xt):
    run(19, 8, 2, 128, 128, 16, xt=xt, in_place=True, drop=0.3)
    run(19, 8, 2, 128, 96, 16, xt=xt, in_place=True, interleaved=True)


def test_unaligned_rows():
    """Heads that start at any element, in tokens and heads of any stride."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, H, D = 6, 2, 64
    k, v = (torch.randn(T * 140 + 5, generator=g, device="cuda").bfloat16()[i:i + T * 140].view(T, 2, 70)[..., :D]
            for i in (1, 3))
    kc, vc = (torch.zeros(3, 4, H, 66, device="cuda", dtype=BF16)[..., 1:1 + D] for _ in range(2))
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 1000
    f = torch.logspace(0, -3, D // 2, device="cuda")
    slots = torch.arange(T, device="cuda", dtype=torch.int32) + 5
    q = k.clone()
    fb.moe_ffn_append_kv(k, v, pos, slots, f, kc, vc, q=q)
    want, err = turned(k, pos, f, False, 1.0)
    close(kc.reshape(12, H, D)[5:11], want, err)
    close(q, want, err)
    assert torch.equal(vc.reshape(12, H, D)[5:11], v)
    assert float(kc.reshape(12, H, D)[:5].abs().max()) == 0 and float(kc.reshape(12, H, D)[11:].abs().max()) == 0


@pytest.mark.parametrize("value", [256.0, -1000.0, float("inf"), float("nan")])
def test_a_frequency_out_of_range_gives_nan(value):
    k = torch.ones(2, 1, 8, device="cuda")
    kc, vc = torch.zeros(1, 4, 1, 8, device="cuda"), torch.zeros(1, 4, 1, 8, device="cuda")
    f = torch.tensor([0.5, value, -255.0, 1e-40], device="cuda")
    pos, slots = torch.tensor([3, 70000], device="cuda", dtype=torch.int32), torch.tensor([0, 2], device="cuda", dtype=torch.int32)
    fb.moe_ffn_append_kv(k, k, pos, slots, f, kc, vc)
    bad = torch.tensor([False, True, False, False] * 2, device="cuda")
    assert bool(kc[0, [0, 2]][..., bad].isnan().all()) and not bool(kc[0, [0, 2]][..., ~bad].isnan().any())
    f[1] = 0.25
    want, err = turned(k, pos, f, False, 1.0)
    close(kc[0, [0, 2]][..., ~bad], want[..., ~bad], err[..., ~bad])


def test_slots_out_of_range_write_nothing():
    """Slots below 0 and from the last page's end on, with memory on both sides of the cache that has to stay."""
    full = torch.full((5, 4, 2, 16), 9.0, device="cuda", dtype=BF16)
    kc, vc = full[1:4], torch.full((3, 4, 2, 16), 9.0, device="cuda", dtype=BF16)
    T = 5
    k, q = torch.ones(T, 2, 16, device="cuda", dtype=BF16), torch.full((T, 2, 16), 2.0, device="cuda", dtype=BF16)
    slots = torch.tensor([-1, 12, -(2**31), 2**31 - 1, 11], device="cuda", dtype=torch.int32)
    fb.moe_ffn_append_kv(k, k, torch.zeros(T, device="cuda", dtype=torch.int32), slots, None, kc, vc, q=q)
    assert float((full == 1).sum()) == 32 and bool((kc[2, 3] == 1).all()) and float((full == 9).sum()) == 18 * 32 + 32
    assert float((vc == 1).sum()) == 32
    assert bool((q == 2).all())  # rot 0: queries as they are


def test_large_offsets():
    """Places in a cache past 2^31 elements."""
    H, D, page = 2, 64, 16
    pages = 2**31 // (page * H * D) + 9
    if torch.cuda.mem_get_info()[0] < 20 * 2**30:
        pytest.skip("needs 10 GB")
    kc, vc = torch.empty(pages, page, H, D, device="cuda", dtype=BF16), torch.empty(pages, page, H, D, device="cuda", dtype=BF16)
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(3, H, D, generator=g, device="cuda").bfloat16()
    slots = torch.tensor([(pages - 1) * page + 15, 0, (pages - 4) * page], device="cuda", dtype=torch.int32)
    fb.moe_ffn_append_kv(k, k, torch.zeros(3, device="cuda", dtype=torch.int32), slots, torch.ones(D // 2, device="cuda"), kc, vc)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, s % page], k[t]) and torch.equal(vc[s // page, s % page], k[t])


@pytest.mark.parametrize("T", [1, 50])
def test_repeats_graphs_and_streams(T):
    g = torch.Generator(device="cuda").manual_seed(T)
    k, q = torch.randn(T, 2, 64, generator=g, device="cuda").bfloat16(), torch.randn(T, 8, 64, generator=g, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + 90000
    f = torch.logspace(0, -4, 32, device="cuda")
    new = lambda: (torch.zeros(8, 8, 2, 64, device="cuda", dtype=BF16), torch.zeros(8, 8, 2, 64, device="cuda", dtype=BF16),  # noqa: E731
                   torch.zeros_like(q))
    want = new()
    fb.moe_ffn_append_kv(k, k, pos, pos - 90000, f, want[0], want[1], q=q, q_out=want[2])
    got = new()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    slots = pos - 90000
    torch.cuda.synchronize()
    fb.moe_ffn_append_kv(k, k, pos, slots, f, got[0], got[1], q=q, q_out=got[2], stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.moe_ffn_append_kv(k, k, pos, slots, f, got[0], got[1], q=q, q_out=got[2])
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("xt,ct,interleaved,in_place", [(BF16, BF16, False, False), (F16, F16, True, True), (F32, BF16, False, True),
                                                        (F32, F32, True, False)])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page", [
    (4096, 32, 4, 128, 128, 16), (2003, 64, 8, 128, 64, 64), (20011, 4, 2, 64, 64, 128), (5003, 14, 2, 96, 48, 24),
    (9001, 6, 1, 36, 20, 7), (7001, 2, 1, 512, 512, 8)])
def test_many_tokens_a_block(T, Hq, Hkv, D, rot, page, xt, ct, interleaved, in_place):
    """Every block takes tokens one behind the other, more of them than lie in its ring, padding among them; heads
    of more items than a block has threads are shared by several."""
    run(T, Hq, Hkv, D, rot, page, xt=xt, ct=ct, qt=ct, interleaved=interleaved, in_place=in_place, layout="head" if in_place else "token",
        drop=0.1, first=70000, scale=0.75)

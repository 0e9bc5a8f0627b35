"""What the binding does with its arguments before it calls the library, on the host: a library that records the call
stands in for the real one."""

import ctypes

import pytest

import fusion_backend_gb300 as fb

torch = pytest.importorskip("torch")


class Recorder:
    """Takes any call, keeps its arguments (argument blocks by value) and returns OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, [type(a).from_buffer_copy(a) if isinstance(a, ctypes.Structure) else a for a in args]))
            return fb.OK

        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(fb, "_lib", r)
    monkeypatch.setattr(fb, "_blocks", {})
    monkeypatch.setattr(fb, "_on_device", lambda first, **tensors: None)
    # tensors on the CPU pass for tensors on the current device
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    return r


def test_a_number_held_in_a_tensor_is_read_on_every_call(rec):
    r, n, alpha = torch.zeros(3, 8), torch.zeros(3, 8), torch.tensor(0.5)
    fb.moe_ffn_norm_residual(r, alpha=alpha, normed=n, stream=1)
    alpha.fill_(2.0)
    fb.moe_ffn_norm_residual(r, alpha=alpha, normed=n, stream=1)
    assert [c[1][0].alpha for c in rec.calls] == [0.5, 2.0]
    lg, ids, w = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    scale = torch.tensor(1.5)
    for v in (1.5, 3.0):
        scale.fill_(v)
        fb.moe_ffn_route(lg, 2, scale=scale, ids=ids, weights=w, stream=1)
    assert [c[1][0].scale for c in rec.calls[2:]] == [1.5, 3.0]


def test_numbers_of_equal_value_find_one_block(rec):
    r, n = torch.zeros(3, 8), torch.zeros(3, 8)
    for alpha in (0.5, 0.5, 1.0, 0.5):
        fb.moe_ffn_norm_residual(r, alpha=alpha, normed=n, stream=1)
    assert [c[1][0].alpha for c in rec.calls] == [0.5, 0.5, 1.0, 0.5] and len(fb._blocks) == 2


def test_numbers_past_32_bits_are_refused(rec):
    lg = torch.zeros(1, 8)
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_route(lg.expand(2**32 + 1, 8), 2, stream=1)
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_route(lg, 2**32 + 2, stream=1)
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_norm_residual(torch.zeros(1, 1).expand(2**32 + 1, 1), stream=1)
    bf = torch.bfloat16
    a, b = torch.zeros(1, 1, 8, dtype=bf), torch.zeros(1, 1, 1, dtype=bf)
    T = 2**32 + 1
    x, y = torch.zeros(1, 8, dtype=bf).expand(T, 8), torch.zeros(1, 1).expand(T, 1)
    ids = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fb.moe_ffn_add_adapters(y, x, ids.expand(T), a, b, stream=1)
    with pytest.raises(ValueError, match="32 bits"):
        fb.moe_ffn_adapters_workspace(2**32 + 1, 64, 64, 8)
    assert rec.calls == []


# ---- the layer for a given routing


def layer(T=2, H=256, E=8, k=2, I=16, Is=24, act=fb.ACT_BF16, wfmt=fb.W_BF16):
    m = fb.MoeFFN.__new__(fb.MoeFFN)
    m.plan, m.shapes, m.act, m.wfmt = None, fb.Shapes(T, H, E, k, I, Is), act, wfmt
    m.workspace, m.workspace_bytes = torch.zeros(256, dtype=torch.uint8), 256
    return m


def tensors(m):
    s, bf = m.shapes, torch.bfloat16
    row = {fb.W_BF16: 2 * s.H, fb.W_Q4B32: s.H // 2 + s.H // 16, fb.W_I8: s.H + 16}[m.wfmt]
    raw = (lambda n: torch.zeros(n, 3, s.H, dtype=bf)) if m.wfmt == fb.W_BF16 else (
        lambda n: torch.zeros(n, 3, row, dtype=torch.uint8))
    return dict(x=torch.zeros(s.T, s.H, dtype=torch.float32 if m.act == fb.ACT_F32 else bf),
                ids=torch.zeros(s.T, s.top_k, dtype=torch.int32), weights=torch.zeros(s.T, s.top_k),
                expert_w=raw(s.E * s.I), shexp_w=raw(s.Is), shexp_gate_w=torch.zeros(s.H, dtype=bf),
                out=torch.zeros(s.T, s.H))


@pytest.mark.parametrize("act", [fb.ACT_BF16, fb.ACT_F32])
@pytest.mark.parametrize("wfmt", [fb.W_BF16, fb.W_Q4B32, fb.W_I8])
def test_routed_takes_the_plans_tensors(rec, act, wfmt):
    m = layer(act=act, wfmt=wfmt)
    t = tensors(m)
    m.routed(**t, stream=1)
    m.routed(**{**t, "shexp_w": None, "shexp_gate_w": None}, stream=1)
    m.routed(**{**t, "shexp_gate_w": None}, stream=1)
    # the same bytes under another name, in another shape, and weights inside a larger buffer
    raw = {n: t[n].view(torch.int16) if t[n].dtype == torch.bfloat16 else t[n] for n in t}
    m.routed(**{**raw, "x": raw["x"].view(1, m.shapes.T, m.shapes.H)}, stream=1)
    pool = torch.zeros(t["expert_w"].numel() * t["expert_w"].element_size() + 512, dtype=torch.uint8)
    m.routed(**{**t, "expert_w": pool, "shexp_w": pool}, stream=1)
    # addresses instead of tensors, as the library's own entry takes them
    m.routed(**{**t, "expert_w": t["expert_w"].data_ptr(), "shexp_w": t["shexp_w"].data_ptr(),
                "out": t["out"].data_ptr()}, stream=1)
    if act == fb.ACT_F32:
        m.routed(**{**t, "out": t["x"]}, stream=1)
    assert all(c[0] == "moe_ffn_execute_routed" for c in rec.calls) and len(rec.calls) >= 5


@pytest.mark.parametrize("name,change", [
    ("x", lambda m, t: t["x"][:1]),                                        # another T
    ("x", lambda m, t: t["x"][:, :-8]),                                    # another H
    ("x", lambda m, t: torch.zeros(2, 264, dtype=torch.bfloat16)[:, :256]),  # rows apart
    ("x", lambda m, t: t["x"].half()),
    ("x", lambda m, t: t["x"].float()),
    ("out", lambda m, t: t["out"].bfloat16()),
    ("out", lambda m, t: t["out"].int()),
    ("out", lambda m, t: t["out"][:1]),
    ("out", lambda m, t: torch.zeros(2, 264)[:, :256]),
    ("out", lambda m, t: torch.zeros(256, 2).t()),
    ("expert_w", lambda m, t: t["expert_w"][:-1]),
    ("expert_w", lambda m, t: t["expert_w"].half()),
    ("expert_w", lambda m, t: t["expert_w"].float()),
    ("expert_w", lambda m, t: t["expert_w"].transpose(0, 1)),
    ("shexp_w", lambda m, t: t["shexp_w"][:-1]),
    ("shexp_w", lambda m, t: t["shexp_w"].half()),
    ("shexp_gate_w", lambda m, t: t["shexp_gate_w"][:-1]),
    ("shexp_gate_w", lambda m, t: t["shexp_gate_w"].float()),
    ("shexp_gate_w", lambda m, t: torch.zeros(512, dtype=torch.bfloat16)[::2]),
])
def test_routed_refuses(rec, name, change):
    m = layer()
    t = tensors(m)
    m.routed(**t, stream=1)  # (a call that passed does not let another one pass)
    with pytest.raises(ValueError, match=name):
        m.routed(**{**t, name: change(m, t)}, stream=1)
    assert len(rec.calls) == 1


@pytest.mark.parametrize("wfmt", [fb.W_Q4B32, fb.W_I8])
def test_routed_refuses_floats_as_coded_weights(rec, wfmt):
    m = layer(wfmt=wfmt)
    t = tensors(m)
    with pytest.raises(ValueError, match="expert_w"):
        m.routed(**{**t, "expert_w": torch.zeros(8, 3, 16, 256, dtype=torch.bfloat16)}, stream=1)


def test_routed_takes_plans_apart(rec):
    """Tensors that one plan takes and another does not."""
    small, large = layer(I=16), layer(I=32)
    small.routed(**tensors(small), stream=1)
    with pytest.raises(ValueError, match="expert_w"):
        large.routed(**tensors(small), stream=1)
    f32 = layer(act=fb.ACT_F32)
    with pytest.raises(ValueError, match="x"):
        f32.routed(**tensors(small), stream=1)
    f32.routed(**tensors(f32), stream=1)


def test_tensors_of_another_device_than_the_current_one(rec, monkeypatch):
    m = layer()
    t = tensors(m)
    bf = torch.bfloat16
    a, b = torch.zeros(1, 8, 256, dtype=bf), torch.zeros(1, 256, 8, dtype=bf)
    calls = [
        lambda: m.routed(**t, stream=1),
        lambda: fb.moe_ffn_route(t["out"], 2, ids=t["ids"], weights=t["weights"], stream=1),
        lambda: fb.moe_ffn_norm_residual(t["out"], normed=t["out"].clone(), stream=1),
        lambda: fb.moe_ffn_add_adapters(t["out"], t["x"], t["ids"][:, 0].clone(), a, b,
                                        workspace=torch.zeros(1 << 20, dtype=torch.uint8), stream=1),
    ]
    for c in calls:
        c()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for c in calls:  # (also where the same call has passed before)
        with pytest.raises(ValueError, match="current"):
            c()
    assert len(rec.calls) == len(calls)

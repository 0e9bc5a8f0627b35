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

"""What the calls allocate for the kernels, which write through raw pointers, under torch default dtypes other than fp32. On
the CPU: the library's calls are replaced by stand-ins that check every buffer that they are given, and write nothing."""
import ctypes

import pytest
import torch

import gated_delta_rule_bounded_b200 as kda

BF, F = torch.bfloat16, torch.float32


class Library:
    """The real library's workspace queries; every other call succeeds without doing anything."""

    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        return getattr(self._real, name) if name.endswith("_bytes") or name == "kda_last_error" else lambda *a: 0


@pytest.fixture(params=[BF, torch.float64], ids=["bf16", "f64"])
def other_default(request, monkeypatch):
    from gated_delta_rule_bounded_b200 import build
    build.build()
    fake = Library(kda.load_library())
    monkeypatch.setattr(kda, "load_library", lambda: fake)
    monkeypatch.setattr(kda, "_cuda", lambda t, name: None)
    monkeypatch.setattr(kda, "_stream", lambda device: ctypes.c_void_p(0))
    kept = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield
    torch.set_default_dtype(kept)


def tokens(B=1, T=70, H=2, K=128, dtype=BF):
    return torch.zeros(B, T, H, K, dtype=dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("packed", [False, True])
def test_gated_delta(other_default, dtype, packed):
    q, v = tokens(dtype=dtype), tokens(H=4, dtype=dtype)
    g = torch.zeros(1, 70, 4, dtype=F)
    cu = torch.tensor([0, 30, 70], dtype=torch.int32) if packed else None
    n = 2 if packed else 1
    out = kda.gated_delta_backward(q, q, v, g, g, None, v, None, cu)
    for m, x in (("dq", q), ("dk", q), ("dv", v), ("dg", g), ("dbeta", g)):
        assert out[m].shape == x.shape and out[m].dtype == x.dtype, m
    assert out["d_initial_state"].dtype == F and out["d_initial_state"].shape == (n, 4, 128, 128)
    o, state = kda.gated_delta_prefill(q, q, v, g, g, None, cu)
    assert o.dtype == dtype and state.dtype == F
    assert kda.gated_delta_decode_step(q[:, :1], q[:, :1], v[:, :1], g[:, :1], g[:, :1], torch.zeros(1, 4, 128, 128, dtype=F)).dtype == dtype


@pytest.mark.parametrize("dtype", [BF, F])
def test_layer_norm(other_default, dtype):
    x, w = torch.zeros(5, 64, dtype=dtype), torch.zeros(64, dtype=F)
    y, mean, rstd = kda.layer_norm(x, w, w)
    assert y.dtype == dtype and mean.dtype == rstd.dtype == F
    out = kda.layer_norm_backward(x, x, w, mean, rstd)
    assert out["dx"].dtype == dtype and out["dweight"].dtype == out["dbias"].dtype == F


@pytest.mark.parametrize("packed", [False, True])
def test_channel_decays(other_default, packed):
    q, gate, beta = tokens(), tokens(dtype=F), torch.zeros(1, 70, 2, dtype=F)
    cu = torch.tensor([0, 30, 70], dtype=torch.int32) if packed else None
    n = 2 if packed else 1
    for call in (kda.scan_backward, kda.scan_backward_chunked):
        out = call(q, q, q, gate, beta, None, q, None, cu)
        for m, x in (("dq", q), ("dk", q), ("dv", q), ("dgate", q), ("dbeta", beta)):
            assert out[m].shape == x.shape and out[m].dtype == F, (call, m)
        assert out["d_initial_state"].shape == (n, 2, 128, 128) and out["d_initial_state"].dtype == F
    o, state = kda.prefill(q, q, q, gate, beta, None, cu)
    assert o.dtype == BF and state.dtype == F
    dz, dA = kda.bounded_decay_backward(gate, torch.zeros(2, dtype=F), -5.0, gate)
    assert dz.dtype == F and dA.dtype == F
    assert kda.bounded_decay(gate, torch.zeros(2, dtype=F)).dtype == F

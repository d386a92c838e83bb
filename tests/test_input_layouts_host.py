"""Inputs whose layout the kernels do not read are copied by the Python calls: rows off 16-byte boundaries. On the CPU: the
library's calls are replaced by stand-ins that keep the pointers and strides they are given, and write nothing."""
import ctypes

import pytest
import torch

import gated_delta_rule_bounded_b200 as kda

BF, F = torch.bfloat16, torch.float32


class Library:
    def __init__(self, real):
        self._real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name == "kda_last_error":
            return getattr(self._real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    from gated_delta_rule_bounded_b200 import build
    build.build()
    fake = Library(kda.load_library())
    monkeypatch.setattr(kda, "load_library", lambda: fake)
    monkeypatch.setattr(kda, "_cuda", lambda t, name: None)
    monkeypatch.setattr(kda, "_stream", lambda device: ctypes.c_void_p(0))
    return fake


def shifted(*shape, dtype=BF):
    """A contiguous tensor one element past a 16-byte boundary."""
    n = 1
    for s in shape:
        n *= s
    t = torch.randn(n + 1).to(dtype)[1:].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


@pytest.mark.parametrize("dtype", [BF, F])
def test_rows_off_a_boundary_are_copied(library, dtype):
    t = shifted(2, 3, 4, 64, dtype=dtype)
    got = kda._rowwise(t)
    assert torch.equal(got, t) and got.data_ptr() % 16 == 0
    every_other = torch.randn(2, 3, 4, 128).to(dtype)[..., ::2]
    assert torch.equal(kda._rowwise(every_other), every_other) and kda._rowwise(every_other).is_contiguous()
    narrow = torch.zeros(2, 3, 5, 1, dtype=dtype)  # rows that no copy would put on boundaries
    assert kda._rowwise(narrow) is narrow
    fine = torch.zeros(2, 3, 4, 64, dtype=dtype)
    assert kda._rowwise(fine) is fine and kda._rowwise(fine[:, :2]).data_ptr() == fine.data_ptr()


@pytest.mark.parametrize("dtype", [BF, F])
def test_every_call_gets_rows_on_boundaries(library, dtype):
    q, v = shifted(1, 70, 2, 64, dtype=dtype), shifted(1, 70, 4, 64, dtype=dtype)
    g = torch.zeros(1, 70, 4)
    kda.gated_delta_prefill(q, q, v, g, g)
    kda.gated_delta_backward(q, q, v, g, g, None, v)
    kda.gated_delta_decode_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], torch.zeros(1, 4, 64, 64))
    gate, beta = shifted(1, 70, 2, 64, dtype=F), torch.zeros(1, 70, 2)
    kda.prefill(q, q, q, gate, beta)
    kda.decode_step(q[:, 0], q[:, 0], q[:, 0], gate[:, 0], beta[:, 0], torch.zeros(1, 2, 64, 64))
    assert len(library.calls) == 5
    for name, args in library.calls:
        for x in args[:3]:
            assert x % 16 == 0, name
    with pytest.raises(ValueError):  # what the call writes is the caller's: not copied, refused
        kda.gated_delta_prefill(q, q, v, g, g, out=shifted(1, 70, 4, 64, dtype=dtype))


def strides(layout, name):
    s = getattr(layout._obj, name)
    return (s.b, s.t, s.h)


@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_expanded_inputs_run_in_chunks(library, which):
    """A stride of zero would send the prefill token by token: the chunked kernels read by TMA, which takes none."""
    x = {"q": torch.randn(2, 100, 2, 64).to(BF), "k": torch.randn(2, 100, 2, 64).to(BF), "v": torch.randn(2, 100, 4, 64).to(BF)}
    x[which] = x[which][:, :, :1].expand_as(x[which])
    g = torch.zeros(2, 100, 4)
    kda.gated_delta_prefill(x["q"], x["k"], x["v"], g, g)
    name, args = library.calls.pop()
    assert name == "kda_gated_delta_prefill" and args[18] and 0 not in strides(args[-5], which)
    # Token by token (no workspace, or fp32) such strides are read as they are.
    kda.gated_delta_prefill(x["q"], x["k"], x["v"], g, g, use_workspace=False)
    assert strides(library.calls.pop()[1][-5], which)[2] == 0
    kda.gated_delta_prefill(x["q"].float(), x["k"].float(), x["v"].float(), g, g)
    assert library.calls.pop()[1][18] is None
    # One token row and one head have no stride that counts.
    kda.gated_delta_prefill(x["q"][:1, :, :1], x["k"][:1, :, :1], x["v"][:1, :, :1], g[:1, :, :1], g[:1, :, :1])
    assert library.calls.pop()[1][0 if which == "q" else 1 if which == "k" else 2] == x[which].data_ptr()

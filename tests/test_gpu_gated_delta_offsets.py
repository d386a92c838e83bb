"""Tensors of more than 2^31 elements: what stands past that offset against the same rows in a call of their own, bit for bit."""
import pytest
import torch

import gated_delta_rule_bounded_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
PAST = (1 << 31) + (1 << 20)


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def unit(*shape):
    x = torch.randn(*shape, device=DEV)
    return (x / x.norm(dim=-1, keepdim=True)).to(BF)


def test_decode_states():
    H = HV = 96
    B = PAST // (HV * 128 * 128) + 1
    q, k, v = unit(B, H, 128), unit(B, H, 128), unit(B, HV, 128)
    g, beta = -torch.rand(B, HV, device=DEV), torch.rand(B, HV, device=DEV)
    state = torch.zeros(B, HV, 128, 128, device=DEV)
    last = torch.randn(2, HV, 128, 128, device=DEV)
    state[-2:] = last
    o = kda.gated_delta_decode_step(q, k, v, g, beta, state)
    alone = kda.gated_delta_decode_step(q[-2:], k[-2:], v[-2:], g[-2:], beta[-2:], last)
    torch.cuda.synchronize()
    # The columns' tiles differ with the number of heads, the sums over rows do not.
    assert torch.equal(o[-2:], alone) and torch.equal(state[-2:], last)


def test_prefill_rows():
    B, H, HV, V = 2, 1, 128, 128
    T = PAST // (B * HV * V) + 1
    q, k = unit(B, T, H, 128), unit(B, T, H, 128)
    v = torch.empty(B, T, HV, V, device=DEV, dtype=BF).normal_()
    g, beta = -torch.rand(B, T, HV, device=DEV) * 0.1, torch.rand(B, T, HV, device=DEV)
    slots = (T + 63) // 64 * HV * 25600
    ws = torch.empty(B * slots, device=DEV, dtype=torch.uint8)  # no room for segments: every sequence whole
    o, state = kda.gated_delta_prefill(q, k, v, g, beta, workspace=ws)
    one, s = kda.gated_delta_prefill(q[1:], k[1:], v[1:], g[1:], beta[1:], workspace=ws[:slots])
    torch.cuda.synchronize()
    assert not kda.device_status()
    assert torch.equal(o[1:], one) and torch.equal(state[1:], s)


@pytest.mark.parametrize("D", [128, 16384, 2047])
def test_layer_norm_rows(D):
    rows = PAST // D + 1
    x = torch.empty(rows, D, device=DEV, dtype=BF).normal_()
    y, mean, rstd = kda.layer_norm(x)
    w = torch.ones(D, device=DEV)
    back = kda.layer_norm_backward(x, x, w, mean, rstd)
    z, m, r = kda.layer_norm(x[-300:])
    dx = kda.layer_norm_backward(x[-300:], x[-300:], w, m, r)["dx"]
    torch.cuda.synchronize()
    assert torch.equal(y[-300:], z) and torch.equal(mean[-300:], m) and torch.equal(rstd[-300:], r)
    assert torch.equal(back["dx"][-300:], dx)

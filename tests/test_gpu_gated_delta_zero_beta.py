"""Tokens of write strength zero in the gated delta rule: nothing is written, and the strength still has a gradient, at any
scale of the gradients that come in. Tolerances as in test_gpu_gated_delta.py (2-norms, half steps of 2^-8 in bf16): dq, dk,
dv 2^-7, d_initial_state and dbeta 2^-16, dg 2^-15 of the larger of its norm and its terms'. A power of two on every incoming
gradient changes no rounding of values in the range of normal numbers."""
import pytest
import torch

from tests import gated_delta_fp64 as ref
import gated_delta_rule_bounded_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
TOL = {"dq": 2.0 ** -7, "dk": 2.0 ** -7, "dv": 2.0 ** -7, "dbeta": 2.0 ** -16, "dg": 2.0 ** -15, "d_initial_state": 2.0 ** -16}


def zeroed(T, K, seed):
    d = ref.inputs(1, T, 1, 2, K, K, BF, seed=seed)
    d["beta"][:, ::3] = 0
    d["beta"][:, 70:75] = 0
    return d


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -20, 2.0 ** -50])
def test_gradients_at_every_scale(scale):
    d = zeroed(150, 64, 3)
    want = ref.gradients(d["q"], d["k"], d["v"], d["g"], d["beta"], d["s0"], d["d_o"], d["d_sf"])
    x = {m: t.to(DEV) for m, t in d.items()}
    got = kda.gated_delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["d_o"] * scale, x["d_sf"] * scale)
    torch.cuda.synchronize()
    assert not kda.device_status()
    terms = want.pop("dg_terms").norm().item()
    zero = d["beta"] == 0
    for m, w in want.items():
        g = got[m].double().cpu() / scale
        norm = max(w.norm().item(), terms) if m == "dg" else w.norm().item()
        assert (g - w).norm().item() <= TOL[m] * norm, m
    g, w = got["dbeta"].double().cpu()[zero] / scale, want["dbeta"][zero]
    assert (g - w).norm().item() <= TOL["dbeta"] * w.norm().item()
    assert not got["dv"].cpu()[zero].any()


@pytest.mark.parametrize("T", [5, 64, 150, 1600])
def test_nothing_is_written(T):
    d = ref.inputs(1, T, 1, 2, 128, 128, BF, seed=T)
    x = {m: t.to(DEV) for m, t in d.items()}
    zero = torch.zeros_like(x["beta"])
    o, state = kda.gated_delta_prefill(x["q"], x["k"], x["v"], x["g"], zero)
    torch.cuda.synchronize()
    assert not kda.device_status()
    assert not o.any() and not state.any()

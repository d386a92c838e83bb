"""bf16 outputs of the gated delta rule carry the rounding of the output and nothing of its size beside it.

An element may be off by half a step of bf16, 2^-8 of its value, and by what the value was off before it was rounded.
Operands that are not inputs enter the products in two bf16 parts: 2^-16 of them is left at most, uniform in size, so
2^-16 / sqrt(3) in the root of the mean square, and the errors of a sum's terms are independent. At most six such operands
stand between the inputs and an output (the state, R, Z, U, A and once more the state's update), each in a sum whose terms
have a norm of up to three times the result's (sums of unit rows with random signs): sqrt(6) 3 2^-16 / sqrt(3) = 4.2 2^-16
of the outputs' rms in the root of the mean square; the largest of a million normal errors is 4.9 times that: 21 2^-16,
below 2^-11 of the rms. One operand with its high part alone is off by 2^-8 / sqrt(3) / 1.4 of its terms, the largest by
five times that: 2^-6.
"""
import pytest
import torch

from tests import gated_delta_fp64 as ref
import gated_delta_rule_bounded_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def rounded(got, want, what):
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    rms = want.square().mean().sqrt()
    over = ((got - want).abs() - 2.0 ** -8 * want.abs()).max().item()
    assert over <= 2.0 ** -11 * rms.item(), f"{what}: an element is {over / rms.item():.3g} of the rms beyond its rounding"


CASES = [  # B, T, H, HV, K, V, packed offsets
    (1, 64, 1, 2, 128, 128, None), (2, 200, 2, 2, 128, 128, None), (1, 333, 1, 3, 128, 128, None), (1, 130, 1, 2, 128, 256, None),
    (1, 97, 2, 2, 48, 80, None), (1, 300, 2, 4, 64, 64, (3, 70, 70, 71, 200, 299)), (1, 1601, 1, 1, 128, 128, None),
    (1, 1800, 1, 2, 64, 128, (0, 1500, 1503, 1800)), (1, 40, 1, 1, 256, 128, None),
]


@pytest.mark.parametrize("B,T,H,HV,K,V,cuts", CASES)
@pytest.mark.parametrize("q_scale", [1.0, 16.0])
def test_outputs(B, T, H, HV, K, V, cuts, q_scale):
    n = B if cuts is None else len(cuts) - 1
    d = ref.inputs(B, T, H, HV, K, V, BF, seed=T + V, n_states=n)
    d["q"] = d["q"] * q_scale  # a power of two: the rounding is the same, the outputs are larger
    o, sf = ref.scan(d["q"], d["k"], d["v"], d["g"], d["beta"], d["s0"], cuts)
    x = {m: t.to(DEV) for m, t in d.items()}
    cu = None if cuts is None else torch.tensor(cuts, device=DEV, dtype=torch.int32)
    got, _ = kda.gated_delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], cu)
    torch.cuda.synchronize()
    assert not kda.device_status()
    a, b = (0, T) if cuts is None else (cuts[0], cuts[-1])
    rounded(got[:, a:b], o[:, a:b], "o")


GRADS = [  # B, T, H, HV, K, V, packed offsets
    (1, 64, 1, 2, 128, 128, None), (2, 200, 2, 2, 128, 128, None), (1, 333, 1, 3, 128, 128, None), (1, 97, 2, 2, 64, 32, None),
    (1, 300, 2, 4, 64, 64, (3, 70, 70, 71, 200, 299)), (1, 1500, 1, 1, 64, 64, None),
]


@pytest.mark.parametrize("B,T,H,HV,K,V,cuts", GRADS)
def test_gradients(B, T, H, HV, K, V, cuts):
    n = B if cuts is None else len(cuts) - 1
    d = ref.inputs(B, T, H, HV, K, V, BF, seed=T + V, n_states=n)
    want = ref.gradients(d["q"], d["k"], d["v"], d["g"], d["beta"], d["s0"], d["d_o"], d["d_sf"], cuts)
    x = {m: t.to(DEV) for m, t in d.items()}
    cu = None if cuts is None else torch.tensor(cuts, device=DEV, dtype=torch.int32)
    got = kda.gated_delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["d_o"], x["d_sf"], cu)
    torch.cuda.synchronize()
    assert not kda.device_status()
    for m in ("dq", "dk", "dv"):
        rounded(got[m], want[m], m)

"""Tokens of write strength zero in the gated delta rule: nothing is written."""
import pytest
import torch

from tests import gated_delta_fp64 as ref
import gated_delta_rule_bounded_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [5, 64, 150, 1600])
def test_nothing_is_written(T):
    d = ref.inputs(1, T, 1, 2, 128, 128, BF, seed=T)
    x = {m: t.to(DEV) for m, t in d.items()}
    zero = torch.zeros_like(x["beta"])
    o, state = kda.gated_delta_prefill(x["q"], x["k"], x["v"], x["g"], zero)
    torch.cuda.synchronize()
    assert not kda.device_status()
    assert not o.any() and not state.any()

"""The gradient of a layer norm's bias where there is no weight. dbias is a sum of d_y over rows, at most 1000 rows in 592
partial sums: within 2^-18 of the terms' norm in fp32 (a dozen roundings of 2^-24), in bf16 its own rounding, 2^-8."""
import pytest
import torch

import gated_delta_rule_bounded_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("shape", [(1000, 128), (3, 7, 250), (5, 2047), (2, 12288), (0, 64)])
@pytest.mark.parametrize("dt,bt", [(BF, BF), (BF, F), (F, F)])
def test_bias_alone(shape, dt, bt):
    gen = torch.Generator(device=DEV).manual_seed(shape[-1])
    x, dy = (torch.randn(*shape, device=DEV, generator=gen).to(dt) for _ in range(2))
    b = torch.randn(shape[-1], device=DEV, generator=gen).to(bt)
    _, mean, rstd = kda.layer_norm(x, None, b)
    got = kda.layer_norm_backward(dy, x, None, mean, rstd, bias=b)
    ones = kda.layer_norm_backward(dy, x, torch.ones_like(b), mean, rstd)
    torch.cuda.synchronize()
    assert got["dweight"] is None and got["dbias"].dtype == bt and got["dbias"].shape == b.shape
    lead = tuple(range(len(shape) - 1))
    want, terms = dy.double().sum(lead), dy.double().square().sum(lead).sqrt()
    tol = 2.0 ** -18 if bt == F else 2.0 ** -8 * (1 + 2.0 ** -8)
    assert (got["dbias"].double() - want).norm() <= tol * torch.maximum(terms, want.abs()).norm()
    assert torch.equal(got["dx"], ones["dx"]) and torch.equal(got["dbias"], ones["dbias"])
    none = kda.layer_norm_backward(dy, x, None, mean, rstd, bias=b, weight_grads=False)
    assert none["dbias"] is None and torch.equal(none["dx"], got["dx"])
    assert kda.layer_norm_backward(dy, x, None, mean, rstd)["dbias"] is None


def test_refusals():
    x = torch.randn(4, 64, device=DEV)
    _, mean, rstd = kda.layer_norm(x)
    for b in (torch.ones(63, device=DEV), torch.ones(64, device=DEV, dtype=BF), torch.ones(64)):
        with pytest.raises(ValueError):
            kda.layer_norm_backward(x, x, None, mean, rstd, bias=b)
    with pytest.raises(TypeError):
        kda.layer_norm_backward(x.bfloat16(), x.bfloat16(), torch.ones(64, device=DEV), mean, rstd,
                                bias=torch.ones(64, device=DEV, dtype=BF))

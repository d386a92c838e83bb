"""Gradients of the gated delta rule as a training step calls them: more full chunks than the persistent kernel has blocks,
and inputs that are slices of one projection. All heads bit for bit against calls of one query head each (in which a block
has one unit at most; without room for segments, so that both run whole sequences), the shorter ones against fp64. An element
of dq, dk and dv is off by its rounding (2^-8 of its value) and 2^-11 of the rms at most, dbeta and d_initial_state by 2^-16
and dg by 2^-15 in the 2-norm, as in test_gpu_gated_delta_rounding.py and test_gpu_gated_delta.py."""
import pytest
import torch

from tests import gated_delta_fp64 as ref
import gated_delta_rule_bounded_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
NAMES = ("q", "k", "v", "g", "beta")


def whole(x, T, H, HV):
    """The gradients in a workspace that has no room for segments."""
    args = [x[m] for m in NAMES] + [x["s0"], x["d_o"], x["d_sf"]]
    full = kda.gated_delta_backward_workspace_bytes(1, T, H, HV, 128, 128)
    try:
        return kda.gated_delta_backward(*args, workspace=torch.empty(full - 16, device=DEV, dtype=torch.uint8))
    except kda.KDAError:  # nothing to split
        return kda.gated_delta_backward(*args, workspace=torch.empty(full, device=DEV, dtype=torch.uint8))


def of_head(x, h, rep):
    q, v = slice(h, h + 1), slice(h * rep, (h + 1) * rep)
    return {"q": x["q"][:, :, q], "k": x["k"][:, :, q], "v": x["v"][:, :, v], "d_o": x["d_o"][:, :, v], "g": x["g"][:, :, v],
            "beta": x["beta"][:, :, v], "s0": x["s0"][:, v].contiguous(), "d_sf": x["d_sf"][:, v].contiguous()}


def against_fp64(got, want, terms):
    for m, w in want.items():
        g = got[m].double().cpu()
        if m in ("dq", "dk", "dv"):
            assert ((g - w).abs() - 2.0 ** -8 * w.abs()).max() <= 2.0 ** -11 * w.square().mean().sqrt(), m
        else:
            norm = max(w.norm().item(), terms) if m == "dg" else w.norm().item()
            assert (g - w).norm().item() <= 2.0 ** (-15 if m == "dg" else -16) * norm, m


@pytest.mark.parametrize("T,H,HV", [(1280, 24, 24), (1280, 24, 48), (1000, 30, 30)])
def test_many_chunks_a_block(T, H, HV):
    assert (T // 64) * H > 3 * 148 or T == 1000  # 480 full chunks; or 450 and 30 of 40 tokens
    d = ref.inputs(1, T, H, HV, 128, 128, BF, seed=H + HV)
    x = {m: t.to(DEV) for m, t in d.items()}
    got, rep = whole(x, T, H, HV), HV // H
    torch.cuda.synchronize()
    assert not kda.device_status()
    for h in range(H):
        one = whole(of_head(x, h, rep), T, 1, rep)
        v = slice(h * rep, (h + 1) * rep)
        for m in ("dq", "dk"):
            assert torch.equal(got[m][:, :, h:h + 1], one[m]), (m, h)
        for m in ("dv", "dg", "dbeta"):
            assert torch.equal(got[m][:, :, v], one[m]), (m, h)
        assert torch.equal(got["d_initial_state"][:, v], one["d_initial_state"]), h
    if T > 1000:  # fp64 token by token takes long; calls of one head are compared with it elsewhere too
        return
    h = H // 2
    s = of_head(d, h, rep)
    want = ref.gradients(*(s[m] for m in NAMES), s["s0"], s["d_o"], s["d_sf"])
    terms = want.pop("dg_terms").norm().item()
    v = slice(h * rep, (h + 1) * rep)
    against_fp64({m: got[m][:, :, h:h + 1] if m in ("dq", "dk") else got[m][:, v] if m == "d_initial_state" else got[m][:, :, v]
                  for m in want}, want, terms)


@pytest.mark.parametrize("B,T,H,HV,cuts", [(2, 150, 2, 4, None), (1, 333, 3, 3, None), (1, 200, 2, 2, (0, 70, 70, 200)), (1, 1500, 1, 2, None)])
def test_slices_of_one_projection(B, T, H, HV, cuts):
    n = B if cuts is None else len(cuts) - 1
    d = ref.inputs(B, T, H, HV, 128, 128, BF, seed=T, n_states=n)
    x = {m: t.to(DEV) for m, t in d.items()}
    cu = None if cuts is None else torch.tensor(cuts, device=DEV, dtype=torch.int32)
    dense = kda.gated_delta_backward(*(x[m] for m in NAMES), x["s0"], x["d_o"], x["d_sf"], cu)
    row = torch.cat([x[m].flatten(2) for m in ("q", "k", "v")], -1)
    q, k, v = (t.unflatten(-1, (-1, 128)) for t in row.split([128 * H, 128 * H, 128 * HV], -1))
    gb = torch.stack([x["g"], x["beta"]], -1)
    d_o = x["d_o"].transpose(1, 2).contiguous().transpose(1, 2)  # heads first
    got = kda.gated_delta_backward(q, k, v, gb[..., 0], gb[..., 1], x["s0"], d_o, x["d_sf"], cu)
    torch.cuda.synchronize()
    assert not kda.device_status()
    for m in got:
        assert torch.equal(got[m], dense[m]), m
    if T > 1000:
        return
    want = ref.gradients(*(d[m] for m in NAMES), d["s0"], d["d_o"], d["d_sf"], cuts)
    against_fp64(got, {m: w for m, w in want.items() if m != "dg_terms"}, want["dg_terms"].norm().item())


@pytest.mark.parametrize("T,H,HV", [(640, 48, 96)])
def test_prefill_of_many_heads(T, H, HV):
    """More chains than SMs, and value heads on shared query heads, bit for bit against one query head at a time."""
    d = ref.inputs(1, T, H, HV, 128, 128, BF, seed=9)
    x = {m: t.to(DEV) for m, t in d.items()}

    def run(x, H, HV):
        least = (T // 64) * HV * 25600  # every sequence whole
        return kda.gated_delta_prefill(*(x[m] for m in NAMES), x["s0"], workspace=torch.empty(least, device=DEV, dtype=torch.uint8))

    o, state = run(x, H, HV)
    for h in range(H):
        one, s = run(of_head(x, h, 2), 1, 2)
        assert torch.equal(o[:, :, 2 * h:2 * h + 2], one) and torch.equal(state[:, 2 * h:2 * h + 2], s), h
    torch.cuda.synchronize()
    assert not kda.device_status()

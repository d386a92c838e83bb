"""Packed calls of many short sequences: which kernels they run on goes by all their tokens, not by the tokens times the
number of sequences (no GPU needed to ask), and the results there (GPU)."""
import pytest
import torch

from tests import gated_delta_fp64 as ref
import gated_delta_rule_bounded_b200 as kda

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_delta_rule_bounded_b200 import build
    build.build()


@pytest.mark.parametrize("n,each,H,HV,chunked", [
    # One token of each user, and a few of each: token by token. Measured, token by token and chunked: 40 users of 32 heads
    # 47 and 119 us, 64 users with 4 tokens of 96 heads 296 and 529, 8 users with 4 tokens of 32 heads 15 and 28.
    (40, 1, 16, 32, False), (16, 2, 16, 32, False), (8, 4, 16, 32, False), (64, 4, 96, 96, False), (100, 1, 4, 8, False),
    # Prompts: 40 of 32 tokens 240 and 128 us, 2 of 32 tokens and 96 heads 45 and 28.
    (40, 32, 16, 32, True), (2, 32, 96, 96, True), (7, 100, 1, 2, True)])
def test_choice(n, each, H, HV, chunked):
    assert (kda.gated_delta_prefill_workspace_bytes(1, n * each, H, HV, 128, 128, n) > 0) == chunked


def test_dense_calls_choose_as_they_did():
    need = lambda B, T, HV: kda.gated_delta_prefill_workspace_bytes(B, T, HV, HV, 128, 128) > 0  # noqa: E731
    assert not need(64, 8, 32) and need(64, 9, 32) and not need(1, 44, 32) and need(1, 45, 32) and need(1, 32, 96)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,HV,K,V", [([1] * 60, 4, 8, 128, 128), ([2, 0, 1, 3] * 12, 8, 32, 64, 128), ([0] * 5 + [40], 1, 2, 128, 48)])
def test_results(lens, H, HV, K, V):
    cuts = [3]
    for x in lens:
        cuts.append(cuts[-1] + x)
    T, n = cuts[-1] + 2, len(lens)
    # The last case has 45 tokens and little else: one more than the 44 that go token by token for lack of other work.
    chunked = kda.gated_delta_prefill_workspace_bytes(1, T, H, HV, K, V, n) > 0
    assert chunked == (T == 45)
    d = ref.inputs(1, T, H, HV, K, V, BF, seed=n, n_states=n)
    o, sf = ref.scan(d["q"], d["k"], d["v"], d["g"], d["beta"], d["s0"], cuts)
    x = {m: t.cuda() for m, t in d.items()}
    cu = torch.tensor(cuts, device="cuda", dtype=torch.int32)
    out = torch.full(x["v"].shape, 7.0, device="cuda", dtype=BF)
    state = x["s0"].clone()
    kda.gated_delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state, cu, out=out, final_state=state)
    torch.cuda.synchronize()
    a, b = cuts[0], cuts[-1]
    assert (out[:, :a] == 7.0).all() and (out[:, b:] == 7.0).all()
    off = lambda got, want: ((got.double().cpu() - want).norm() / want.norm()).item()  # noqa: E731
    assert off(out[:, a:b], o[:, a:b]) <= 2.0 ** -8  # its own rounding
    # Sums of at most 128 terms in fp32, as every fp32 call's; in chunks, operands in two bf16 parts.
    assert off(state, sf) <= (2.0 ** -16 if chunked else 2.0 ** -18)

"""Outputs that overlap an input in part, or themselves, are refused before a launch (no GPU needed)."""
import ctypes

import pytest

import gated_delta_rule_bounded_b200 as kda
from gated_delta_rule_bounded_b200 import Layout, Strides

OK, INVALID = 0, 1
FAKE = 1 << 30  # a non-null, 16-byte aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_bounded_b200 import build
    build.build()
    return kda.load_library()


ROWS, D = 4, 64  # bf16: rows of 128 bytes


@pytest.mark.parametrize("xs,y", [
    (64, FAKE + 128), (64, FAKE - 128), (64, FAKE + 2), (64, FAKE + 3 * 128 + 64),  # shifted by rows, by elements, the last half row
    (128, FAKE), (128, FAKE + 128), (0, FAKE), (32, FAKE),  # x is not contiguous: its rows are not y's
    (512, FAKE + 1024 - 64), (512, FAKE + 2 * 1024 - 256),  # from between two rows into the next
])
def test_norm_refuses(lib, xs, y):
    assert lib.kda_layer_norm(FAKE, xs, kda.KDA_BF16, None, None, 1, 1e-5, ROWS, D, y, BIG, BIG + 4096, None) == INVALID
    assert "overlap" in lib.kda_last_error().decode()
    for dy, x, dys, xs_ in ((FAKE, BIG, xs, 64), (BIG, FAKE, 64, xs)):  # dx over d_y, and over x
        assert lib.kda_layer_norm_backward(dy, dys, x, xs_, kda.KDA_BF16, None, 1, 2 * BIG, 2 * BIG + 4096, ROWS, D, y, None, None,
                                           None, 0, None) == INVALID
        assert "overlap" in lib.kda_last_error().decode()


@pytest.mark.parametrize("xs,y", [(64, FAKE), (64, FAKE + 512), (64, FAKE - 512), (512, FAKE + 128), (512, FAKE + 1024 + 512),
                                  (512, FAKE + 2 * 1024 + 128)])
def test_norm_takes(lib, xs, y):
    """Refused for another reason, which is looked at later: a null pointer among the results."""
    assert lib.kda_layer_norm(FAKE, xs, kda.KDA_BF16, None, None, 1, 1e-5, ROWS, D, y, None, BIG, None) == INVALID
    assert "overlap" not in lib.kda_last_error().decode()


@pytest.mark.parametrize("o", [(0, 512, 128), (8192, 0, 128), (8192, 512, 0)])
def test_scan_refuses_outputs_over_one_another(lib, o):
    s = (8192, 512, 128)
    layout = Layout(*(Strides(*x) for x in ((4096, 256, 128), (4096, 256, 128), s, (64, 4, 1), (64, 4, 1), o)))
    rc = lib.kda_gated_delta_prefill(FAKE, FAKE, FAKE, 1, FAKE, FAKE, None, None, None, 0, 2, 16, 2, 4, 128, 128,
                                     ctypes.byref(layout), FAKE, None, 0, None)
    assert rc == INVALID and "o " in lib.kda_last_error().decode()
    if o[1]:
        rc = lib.kda_gated_delta_decode_step(FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 2, 2, 4, 128, 128, ctypes.byref(layout), FAKE, None)
        assert rc == INVALID and "o " in lib.kda_last_error().decode()

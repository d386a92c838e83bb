"""Outputs that overlap an input in part are refused before a launch (no GPU needed)."""
import pytest

import gated_delta_rule_bounded_b200 as kda

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
    (512, FAKE + 1024 - 64), (512, FAKE + 3 * 1024 - 256),  # from between two rows into the next
])
def test_norm_refuses(lib, xs, y):
    assert lib.kda_layer_norm(FAKE, xs, kda.KDA_BF16, None, None, 1, 1e-5, ROWS, D, y, BIG, BIG + 4096, None) == INVALID
    assert "overlap" in lib.kda_last_error().decode()
    for dy, x, dys, xs_ in ((FAKE, BIG, xs, 64), (BIG, FAKE, 64, xs)):  # dx over d_y, and over x
        assert lib.kda_layer_norm_backward(dy, dys, x, xs_, kda.KDA_BF16, None, 1, 2 * BIG, 2 * BIG + 4096, ROWS, D, y, None, None,
                                           None, 0, None) == INVALID
        assert "overlap" in lib.kda_last_error().decode()


@pytest.mark.parametrize("xs,y", [(64, FAKE), (64, FAKE + 512), (64, FAKE - 512), (512, FAKE + 128), (512, FAKE + 1024 + 512),
                                  (512, FAKE + 3 * 1024 + 128)])
def test_norm_takes(lib, xs, y):
    """Refused for another reason, which is looked at later: a null pointer among the results."""
    assert lib.kda_layer_norm(FAKE, xs, kda.KDA_BF16, None, None, 1, 1e-5, ROWS, D, y, None, BIG, None) == INVALID
    assert "overlap" not in lib.kda_last_error().decode()

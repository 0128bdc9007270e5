"""The window that a dense call hands to the C ABI."""
import pytest

import exact_attention_blackwell_tiled_gb300 as fa


@pytest.mark.parametrize("window,want", [
    ((5, 0), (5, 0)), ((-1, 7), (-1, 7)), ((-9, -2), (-1, -1)), ((2 ** 31 - 1, 3), (2 ** 31 - 1, 3)),
    ((2 ** 32, 2 ** 32 + 5), (2 ** 31 - 1, 2 ** 31 - 1)), ((2 ** 31, -2 ** 40), (2 ** 31 - 1, -1))])
def test_window_sides(window, want):
    m = fa._score_mod(False, window, None, 2)
    assert (m.window_left, m.window_right) == want

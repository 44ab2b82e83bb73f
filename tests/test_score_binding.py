"""Values of Score that its C fields cannot hold (no GPU)."""
import pytest

from int2_kv_cache_gb300 import Score


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1])
def test_a_window_past_int32_is_refused(window):
    """It would be taken modulo 2^32: as no window, or as one of five tokens."""
    with pytest.raises(ValueError, match="window"):
        Score(window=window)


@pytest.mark.parametrize("cap", [1e-46, -1e-60])
def test_a_cap_that_rounds_to_none_is_refused(cap):
    with pytest.raises(ValueError, match="cap"):
        Score(cap=cap)


def test_others_are_taken():
    assert Score().window == 0 and Score(window=2 ** 31 - 1).window == 2 ** 31 - 1 and Score(cap=1e-40).cap == 1e-40

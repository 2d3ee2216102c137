"""Host checks of the attention calls at the ends of their ranges (no GPU: they come before any
device work)."""
import pytest

from test_abi import _attend, lib  # noqa: F401


@pytest.mark.parametrize("scale,status", [(3.0e38, 1), (2.4e38, 1), (float("inf"), 1), (float("nan"), 1)])
def test_a_scale_that_overflows_is_refused(lib, scale, status):  # noqa: F811
    """The scores are formed with scale times log2(e): infinity there makes NaN of a score of 0."""
    assert _attend(lib, scale=scale) == status

"""The scales that attention takes: its scores are held as powers of two, so that a scale has to stay finite when it is
multiplied by log2(e)."""
from tests.test_cache import EINVAL, call, lib, struct  # noqa: F401  (lib is a fixture)


def test_scales_whose_power_of_two_form_is_infinite_are_refused(lib):  # noqa: F811
    c = struct()
    for scale in (2.4e38, -2.4e38, 3.4e38):
        assert call(lib, "attend", c, scale=scale) == EINVAL
    # taken (and without rows there is nothing to do)
    for scale in (2e38, -2e38, 0.0, 1e-45):
        assert call(lib, "attend", c, scale=scale, rows=0) == 0

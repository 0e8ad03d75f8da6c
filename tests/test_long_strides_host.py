"""Bounds whose rows overlap are refused, on the host, before any CUDA call: other threads write them, in no order."""
import pytest

from paged_mla_kv_cache_gb300 import binding

from test_long_host import BOUNDS


# (block stride, row stride) of 4 pages of 576 values
@pytest.mark.parametrize("bb,br", [
    (576, 576),            # a page's smallest values are the next one's largest
    (1151, 576), (1152, 577), (1152, 640), (2000, 1425),  # one value of the next page
    (576, 1152), (576, 1728), (576, 2303 - 576), (640, 640 * 3), (640, 640 * 3 + 575),  # all largest values, one page too close
    (0, 576), (0, 4096), (575, 4096), (1, 576), (2 ** 39, 2 ** 39), (2 ** 40, 2 ** 40)])
def test_overlapping_rows_are_refused(cuda_lib, bb, br):
    assert cuda_lib.pmg_call_packed(4, binding.BOUNDS_ARGS.pack(*{**BOUNDS, "bb": bb, "br": br}.values())) == 2

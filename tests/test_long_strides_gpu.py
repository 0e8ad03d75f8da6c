"""Layouts of page bounds that keep rows apart."""
import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import long_reference as ref
from test_long_ops_gpu import bounds_case, same
from test_mla_ops_gpu import BF16, DEV, FP8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


@pytest.mark.parametrize("cdt", [BF16, FP8])
@pytest.mark.parametrize("E", [576, 40])
@pytest.mark.parametrize("layout", ["rows apart", "rows close", "pages apart", "one of many"])
def test_bounds_layouts(cdt, E, layout):
    cache, before, table, seq, ctx = bounds_case([0, 70, 5], [200, 30, 1000], E, 64, cdt, BF16)
    n = cache.shape[0]
    whole = {"rows apart": lambda: torch.full((2, n, E + 8), 7.0, dtype=BF16, device=DEV)[:, :, :E].transpose(0, 1),
             "rows close": lambda: torch.full((2, n, E), 7.0, dtype=BF16, device=DEV).transpose(0, 1),
             "pages apart": lambda: torch.full((n, 3, E), 7.0, dtype=BF16, device=DEV)[:, :2],
             "one of many": lambda: torch.full((n, 2, 3, E), 7.0, dtype=BF16, device=DEV)[:, :, 1]}[layout]
    got = whole()
    got.copy_(before)
    binding.block_bounds(cache, got, table, seq, ctx)
    torch.cuda.synchronize()
    assert same(got, ref.bounds(cache, before, table, seq, ctx))

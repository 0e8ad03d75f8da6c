"""Latent attention where neighbours, leftovers and limits could reach a result: what is in shared memory before a call,
and lengths next to the largest."""
import math

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

from test_mla_ops_gpu import BF16, DEV, F16, decode_case, gen, i32, normal, run_decode

pytestmark = pytest.mark.gpu
SM = 1 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


@pytest.fixture(scope="module")
def ws():
    return binding.new_attention_workspace(DEV)


@pytest.mark.parametrize("src", [BF16, F16])
@pytest.mark.parametrize("heads,q_len", [(5, 1), (20, 1), (40, 1), (24, 2), (3, 7)])
def test_decode_bits_do_not_depend_on_the_call_before(ws, src, heads, q_len):
    """Rows that fill up a group of 16, 32 or 64 are 0, whatever an earlier call left in their place."""
    case = decode_case([700, 65, 3000, 1], heads, q_len, src, src, 64)
    want, lse = run_decode(case, ws)
    q, cache, table, lens, _ = case
    out, got = torch.empty_like(want), torch.empty_like(lse)
    other = (normal(gen(8), 200, 1, 64, 576) * 3000).to(src)
    left, pages, n = torch.empty(200, 1, 64, 512, dtype=src, device=DEV), table[2:3].repeat(200, 1), i32([200] * 200)
    for _ in range(20):
        binding.latent_decode(other, cache, pages, n, left, sm_scale=SM, workspace=ws)
        binding.latent_decode(q, cache, table, lens, out, got, sm_scale=SM, workspace=ws)
        assert torch.equal(out, want) and torch.equal(got, lse)

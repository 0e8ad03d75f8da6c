"""Weights over an e4m3 cache hold what fp16 holds of them, in every pass that multiplies them.

A request's first entry has 2^c times the weight of each of its others, whose values are 1 where the first one's are 0. The
others' weights are one number, off by one rounding, so the result is off by that rounding and its own: 2^-11 each for fp16.
c goes through the weights' significant bits from 1024 to 1117, of 1024 to 2047: 11 bits that no 9 hold."""
import math

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import long_reference as ref
from test_long_ops_gpu import call_shared, new_ws, shared_case
from test_mla_ops_gpu import DEV, F16, FP8, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


@pytest.mark.parametrize("kind,reqs,heads", [("prefix", 4, 16), ("prefix", 64, 128), ("own", 3, 128), ("own", 3, 16), ("decode", 3, 64),
                                             ("decode", 5, 20)])
def test_one_weight_of_many_entries(kind, reqs, heads):
    """64 entries, one tile that no share cuts: a prefix of few rows, of pairs of SMs, own entries behind an empty prefix, and
    plain decode."""
    cache = torch.zeros(1, 64, 576, device=DEV)
    cache[0, 1:, :512] = 1.0
    cache[0, 0, 512] = 1.0
    cache = cache.to(FP8)
    c = 1.0 - torch.arange(reqs * heads, device=DEV).view(reqs, 1, heads) * 37 % 128 / 1024.0
    q = torch.zeros(reqs, 1, heads, 576, device=DEV)
    q[..., 512] = c
    q = q.to(F16)
    out = torch.full((reqs, 1, heads, 512), 7.0, dtype=F16, device=DEV)
    full, none = i32([64]), i32([0])
    table = torch.zeros(reqs, 1, dtype=torch.int32, device=DEV)
    if kind == "decode":
        binding.latent_decode(q, cache, table, i32([64] * reqs), out, sm_scale=math.log(2), workspace=binding.new_attention_workspace(DEV))
    else:
        binding.latent_decode_shared(q, cache, table[:1], full if kind == "prefix" else none, i32([0, reqs]), table,
                                     i32([0 if kind == "prefix" else 64] * reqs), out, sm_scale=math.log(2),
                                     workspace=binding.new_shared_workspace(DEV, reqs, 1, heads, 512))
    w = 63 * 2.0 ** -c.double()
    want = (w / (1 + w))[..., None]
    # scores, exponentials and sums in 32 bits: below 2^-18
    off = (out.double() / want - 1).abs().max()
    assert off <= 2.0 ** -11 * (1 + 2.0 ** -11) + 2.0 ** -11 + 2.0 ** -18, f"off by 2^{math.log2(off):.2f}"


@pytest.mark.parametrize("members,prefix,heads", [([3, 2], [700, 65], 16), ([20, 1, 0, 40], [3001, 5000, 64, 130], 32)])
def test_errors_of_fp16_over_e4m3_together(members, prefix, heads):
    """All values together are off by the rounding of the results and that of the weights, alike in size and not of each other:
    sqrt(2) times what weights in 32 bits leave, and here no more than 1.5 times."""
    c = shared_case(members, prefix, [17] * sum(members), heads, 1, F16, FP8, 64)
    sm = 1 / math.sqrt(192)
    out, lse = torch.empty(c["q"].shape[:3] + (512,), dtype=F16, device=DEV), torch.empty(c["q"].shape[:3], device=DEV)
    call_shared(c, out, lse, sm, new_ws(c))
    want = ref.shared(c["q"], c["cache"], c["ptable"], c["plens"], c["cu"], c["table"], c["lens"], 512, sm, float(c["scale"]))[0]
    least = (want.to(F16).double() - want).norm()
    assert (out.double() - want).norm() <= 1.5 * least, f"{(out.double() - want).norm() / least:.2f} times the results' rounding"

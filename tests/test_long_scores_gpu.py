"""Page scores where their terms are odd or leave no room: infinite bounds, pages of equal entries, entries taken back."""
import math

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import long_reference as ref
from test_long_ops_gpu import same, score_case
from test_mla_ops_gpu import BF16, DEV, F16, F32, GENERAL, gen, i32, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


def score(case, sm, options):
    q, bound, table, lens, block, scale, lse = case
    out, err = torch.full((q.shape[0], q.shape[1], table.shape[1]), 7.0, device=DEV), i32([0])
    binding.block_scores(q, bound, table, lens, out, block_size=block, sm_scale=sm, scale=scale, lse=lse, error_flag=err, options=options)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out.double()


def largest(case, sm):
    """max_h (sm sum_d max(q hi, q lo) - lse) of every page that a token sees, and the largest sum of its finite magnitudes."""
    q, bound, table, lens, block, _, lse = case
    R, n, H, _ = q.shape
    out = torch.full((R, n, table.shape[1]), -math.inf, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    for r in range(R):
        for i in range(n):
            for c in range(-(-max(int(lens[r]) - n + 1 + i, 0) // block)):
                x, (hi, lo) = q[r, i].double(), bound[int(table[r, c])].double()
                terms = torch.maximum(x * hi, x * lo)
                s = terms.sum(1) * sm - lse[r, i].double()
                out[r, i, c] = math.nan if s.isnan().any() else s.max()
                mag[r, i, c] = (torch.where(terms.isfinite(), terms, 0.0).abs().sum(1) * sm + lse[r, i].double().abs()).max()
    return out, mag


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("heads,q_len,dtype", [(16, 1, BF16), (16, 3, F16), (5, 4, BF16), (128, 2, BF16), (100, 1, F16), (1, 1, F16),
                                               (16, 1, F32), (65, 2, BF16)])
def test_scores_of_infinite_bounds(options, heads, q_len, dtype):
    """An infinite entry bounds a head of the other sign by the page's other bound, which is a number: max(q hi, q lo)."""
    case = score_case([700, 70, 5000], heads, q_len, dtype, 64, lse=True)
    q, bound, table = case[:3]
    q[..., 5:40] = torch.where(q[..., 5:40] == 0, 1.0, q[..., 5:40])
    at = lambda r, c: int(table[r, c])  # noqa: E731
    bound[at(0, 0), 0, 7] = math.inf
    bound[at(0, 2), 1, 8] = -math.inf
    bound[at(0, 9), 0, 9], bound[at(0, 9), 1, 9] = math.inf, -math.inf
    bound[at(1, 0), :, 10] = math.inf                                   # every entry is infinite there
    bound[at(2, 63), :, 11], bound[at(2, 64), 0, 12:30] = -math.inf, math.inf
    bound[at(2, 70), :, 13], bound[at(2, 70), :, 14] = -math.inf, math.inf
    q[0, 0, 0, 7], q[:, :, :, 14] = -q[0, 0, 0, 7].abs(), -q[:, :, :, 14].abs()  # one head that the infinity lowers, and all
    q[:, :, :, 10] = -q[:, :, :, 10].abs()                              # nothing but -inf
    got = score(case, 0.07, options)
    want, mag = largest(case, 0.07)
    assert torch.equal(got.isnan(), want.isnan()) and not want.isnan().all()
    odd = ~want.isfinite()
    assert torch.equal(got[odd].nan_to_num(), want[odd].nan_to_num())
    # 2 E products summed in 32 bits; the factor's rounding, its product, the log sum
    err, most = (got - want).abs()[~odd], (((2 * 576 + 72) * 2.0 ** -24) * mag + 1e-30)[~odd]
    assert (err <= most).all(), f"off by {(err / most).max():.3g} of the bound"
    assert want[0].isfinite()[:, 1].all() and (want[1, -1, 0] == -math.inf) and (want == math.inf).any()


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scores_of_a_zero_and_an_infinity(options):
    """0 times an infinity has no value; an infinite query or bound beside numbers has."""
    case = score_case([300, 300], 16, 1, BF16, 64, lse=True)
    q, bound, table = case[:3]
    bound[int(table[0, 1]), 0, 3], bound[int(table[0, 3]), 1, 4] = math.inf, -math.inf
    q[0, 0, 7, 3], q[0, 0, 9, 4] = 0.0, -0.0
    q[1, 0, 5, 6] = math.inf
    got, want = score(case, 0.07, options), largest(case, 0.07)[0]
    assert torch.equal(got.isnan(), want.isnan()) and got[0, 0, [1, 3]].isnan().all() and got[0, 0, [0, 2, 4]].isfinite().all()
    assert (got[1, 0] == math.inf).all()


@pytest.mark.parametrize("dtype,heads", [(F16, 128), (BF16, 16)])
def test_scores_of_nothing_but_infinities(dtype, heads):
    """Every page has columns of both infinities that lower every head: all scores are -inf, and the call ends in time."""
    case = score_case([4096] * 5, heads, 4, dtype, 16, lse=True)
    q, bound = case[:2]
    bound[:, :, 100], bound[:, :, 101] = -math.inf, math.inf
    q[..., 100], q[..., 101] = 1.0 + normal(gen(1), 5, 4, heads).abs().to(dtype), -1.0
    got, want = score(case, 0.07, 0), largest(case, 0.07)[0]
    assert torch.equal(got, want) and (got == -math.inf).all()


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("heads,dtype", [(16, BF16), (128, F16), (128, BF16), (5, F16), (16, F32)])
@pytest.mark.parametrize("block", [1, 64])
@pytest.mark.parametrize("one_sign", [True, False])
def test_scores_of_equal_entries(options, heads, dtype, block, one_sign):
    """Where a page's entries are one, its score is theirs: the bound has no room to hide a lost part of the sum in."""
    pages = 70
    entry = normal(gen(1), pages, 1, 576)
    q = normal(gen(2), 1, 1, heads, 576)
    if one_sign:
        entry, q = entry.abs(), q.abs()
    entry, q = entry.to(dtype), q.to(dtype)
    cache = entry.expand(pages, block, 576).contiguous()
    bound = torch.full((pages, 2, 576), 7.0, dtype=dtype, device=DEV)
    table, lens = torch.randperm(pages, generator=gen(3), device=DEV).to(torch.int32).view(1, pages), i32([pages * block])
    binding.block_bounds(cache, bound, table, lens)
    assert torch.equal(bound, entry.expand(pages, 2, 576))
    case = (q, bound, table, lens, block, None, None)
    got = score(case, 0.07, options)[0, 0]
    terms = q[0, 0].double()[:, None] * entry[table[0].long(), 0].double() * 0.07
    want, mag = terms.sum(2).amax(0), terms.abs().sum(2).amax(0)
    assert ((got - want).abs() <= (2 * 576 + 72) * 2.0 ** -24 * mag).all(), f"off by {((got - want).abs() / mag).max():.3g}"


def test_bounds_after_entries_were_taken_back():
    """Refused drafts widen a begun page's bounds, and leave with the page's first place."""
    cache = normal(gen(1), 3, 64, 576, dtype=BF16)
    bound, table = torch.zeros(3, 2, 576, dtype=BF16, device=DEV), i32([[2, 0, 1]])
    binding.block_bounds(cache, bound, table, i32([60]))
    drafts = cache.clone()
    drafts[2, 61:64], drafts[0, :2] = 50.0, -50.0
    binding.block_bounds(drafts, bound, table, i32([66]), i32([60]))   # six tokens drafted
    assert (bound[2, 0] == 50).all() and (bound[0, 1] == -50).all()
    binding.block_bounds(cache, bound, table, i32([63]), i32([61]))    # one kept, two of the next step
    assert (bound[2, 0] == 50).all() and torch.equal(bound[2, 1], torch.minimum(cache[2, :63].amin(0), drafts[2, 60]))
    binding.block_bounds(cache, bound, table, i32([66]), i32([63]))
    whole = ref.bounds(cache, torch.zeros_like(bound), table, i32([66]))
    assert torch.equal(bound[0], whole[0])                             # begun anew
    assert (bound[2, 0] >= whole[2, 0]).all() and (bound[2, 1] <= whole[2, 1]).all()
    binding.block_bounds(cache, bound, table, i32([64]), i32([0]))
    assert same(bound, whole)

"""The operators for long contexts on the GPU against their 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import long_reference as ref
import mla_reference as mref
from test_mla_ops_gpu import BF16, DEV, F16, F32, FP8, GENERAL, decode_case, gen, i32, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


# --- block_bounds ------------------------------------------------------------------

def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.double().nan_to_num(7.0), b.double().nan_to_num(7.0))


def bounds_case(ctx, new, E, block, cdt, bdt, stride=None, seed=5, gap=0):
    rng = np.random.default_rng(seed)
    g = gen(seed)
    seq = [c + n for c, n in zip(ctx, new)]
    table, blocks = mref.tables(rng, seq, block)
    full = normal(g, blocks, block, stride or E)
    full = ((full * 20).clamp(-448, 448) if cdt == FP8 else full).to(cdt)
    for r, n in enumerate(seq):  # slots past a request's end hold anything
        if n > 0 and n % block:
            full[int(table[r, n // block]), n % block:] = math.nan
    before = torch.full((blocks, 2, E + gap), 7.0, device=DEV).to(bdt)[:, :, :E]
    before.copy_(normal(g, blocks, 2, E).abs() * torch.tensor([[[1.0], [-1.0]]], device=DEV))
    return full[:, :, :E], before, i32(table), i32(seq), i32(ctx)


def run_bounds(case, with_ctx=True, flag=0):
    cache, before, table, seq, ctx = case
    want = ref.bounds(cache, before, table, seq, ctx if with_ctx else None)
    got, err = before.clone() if before.is_contiguous() else before, i32([0])
    binding.block_bounds(cache, got, table, seq, ctx if with_ctx else None, err)
    torch.cuda.synchronize()
    assert int(err) == flag
    assert same(got, want)
    return got


@pytest.mark.parametrize("cdt,bdt", [(BF16, BF16), (F16, F16), (F32, F32), (FP8, BF16), (FP8, F16), (FP8, F32)])
@pytest.mark.parametrize("E,stride,block,gap", [(576, None, 64, 0), (576, 640, 16, 64), (576, 577, 64, 0), (40, None, 7, 3),
                                                (1, None, 3, 0), (1024, None, 8, 0), (300, None, 1, 0), (16, 48, 200, 16)])
def test_bounds(cdt, bdt, E, stride, block, gap):
    case = bounds_case([0, 5, block, 3 * block + 1, 17, 0, 60], [1, 0, 1, 2 * block + 1, 300, 0, 5], E, block, cdt, bdt, stride,
                       gap=gap)
    run_bounds(case)
    run_bounds(case, with_ctx=False)


@pytest.mark.parametrize("reqs", [1, 32, 33, 700])
def test_bounds_many_requests(reqs):
    rng = np.random.default_rng(reqs)
    ctx, new = rng.integers(0, 70, reqs), rng.integers(0, 40, reqs)
    new[::5] = 0
    run_bounds(bounds_case(ctx.tolist(), new.tolist(), 64, 16, BF16, BF16))


def test_bounds_of_steps_are_those_of_the_whole():
    """Entries that join a few at a time leave the bounds of all of them."""
    cache, before, table, seq, ctx = bounds_case([0, 0, 0], [200, 17, 1000], 576, 64, BF16, BF16)
    whole = run_bounds((cache, before, table, seq, ctx), with_ctx=False)
    got, at = before.clone(), torch.zeros_like(seq)
    while (at < seq).any():
        to = (at + 37).minimum(seq)
        binding.block_bounds(cache, got, table, to, at)
        at = to
    assert same(got, whole)


@pytest.mark.parametrize("cdt,bdt", [(BF16, BF16), (F16, F16), (F32, F32), (FP8, BF16)])
@pytest.mark.parametrize("stride", [576, 577])
def test_bounds_of_odd_values(cdt, bdt, stride):
    """NaN makes NaN of its column, new or known before; infinities are values like others."""
    case = bounds_case([0, 70], [130, 30], 576, 64, cdt, bdt, stride)
    cache, before, table, seq, ctx = case
    cache[int(table[0, 1]), 3, 5] = math.nan
    cache[int(table[1, 1]), 20, 9] = math.nan
    before[int(table[1, 1]), 0, 11] = math.nan
    before[int(table[0, 0]), 0, 12] = math.nan  # not begun: forgotten
    if cdt != FP8:
        cache[int(table[0, 0]), 1, 7] = math.inf
        cache[int(table[0, 0]), 2, 7] = -math.inf
    got = run_bounds(case)
    assert got[int(table[0, 1]), :, 5].isnan().all() and got[int(table[1, 1]), :, 9].isnan().all()
    assert got[int(table[1, 1]), 0, 11].isnan() and not got[int(table[0, 0])].isnan().any()


def test_bounds_bad_data():
    case = bounds_case([0, 64, 0, 5], [200, 100, 64, 3], 576, 64, BF16, BF16)
    cache, before, table, seq, ctx = case
    table[0, 1], table[1, 2] = -1, cache.shape[0]
    run_bounds(case, flag=binding.FLAG_PHYS_BLOCK)
    seq[2], ctx[3] = -3, -9
    run_bounds(case, flag=binding.FLAG_PHYS_BLOCK | binding.FLAG_LENGTH)
    seq[0] = table.shape[1] * 64 + 1
    run_bounds(case, flag=binding.FLAG_PHYS_BLOCK | binding.FLAG_LENGTH | binding.FLAG_LOGICAL_BLOCK)


def test_bounds_past_32_bit_offsets():
    blocks, block = 120000, 64  # 4.6e9 elements
    cache = torch.empty(blocks, block, 600, dtype=BF16, device=DEV)[:, :, :576]
    bounds = torch.zeros(blocks, 2, 20000, dtype=BF16, device=DEV)[:, :, :576]  # 4.8e9 elements
    pages = [blocks - 1, 0, 60001, blocks - 7]
    for p in pages:
        cache[p] = normal(gen(p + 1), block, 576, dtype=BF16)
    binding.block_bounds(cache, bounds, i32([pages]), i32([230]), i32([64]))
    for k, p in enumerate(pages):
        rows = cache[p, :230 - 64 * k]
        want = torch.stack([rows.amax(0), rows.amin(0)]) if k else torch.zeros(2, 576, dtype=BF16, device=DEV)
        assert torch.equal(bounds[p], want)


# --- block_scores ------------------------------------------------------------------

def score_case(lens, heads, q_len, dtype, block, E=576, seed=6, lse=False, scale=None, unaligned=0):
    rng = np.random.default_rng(seed)
    g = gen(seed)
    table, blocks = mref.tables(rng, lens, block)
    bound = torch.zeros(blocks, 2, E + unaligned, dtype=dtype, device=DEV)[:, :, unaligned:]
    bound.copy_((2.3 + 0.4 * normal(g, blocks, 2, E)) * torch.tensor([[[1.0], [-1.0]]], device=DEV))
    q = torch.zeros(len(lens), q_len, heads, E + unaligned, dtype=dtype, device=DEV)[..., unaligned:]
    q.copy_(normal(g, len(lens), q_len, heads, E))
    return (q, bound, i32(table), i32(lens), block, None if scale is None else torch.tensor([scale], device=DEV),
            3 + normal(g, len(lens), q_len, heads) if lse else None)


def run_scores(case, sm=0.07, options=0, flag=0, pad=0):
    q, bound, table, lens, block, scale, lse = case
    R, n, H, E = q.shape
    W = table.shape[1]
    out, err = torch.full((R, n, W + pad), 7.0, device=DEV), i32([0])
    binding.block_scores(q, bound, table, lens, out[:, :, :W], block_size=block, sm_scale=sm, scale=scale, lse=lse,
                         error_flag=err, options=options)
    torch.cuda.synchronize()
    assert int(err) == flag and (out[:, :, W:] == 7).all()
    f = sm * (1.0 if scale is None else float(scale))
    want, mag = ref.scores(q, bound, table, lens, block, f, lse)
    got = out[:, :, :W].double()
    finite = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~finite].nan_to_num(), want[~finite].nan_to_num())
    # 2 E products, exact or rounded once, summed in 32 bits; then the factor's own rounding, its product, the log sum
    bound_of = ((2 * E + 64) * 2.0 ** -24 + 8 * 2.0 ** -24) * mag + 1e-30
    err = (got - want).abs()[finite]
    assert (err <= bound_of[finite]).all(), f"off by {err.max():.3g}, {(err / bound_of[finite]).max():.3g} of its bound"
    return out[:, :, :W]


LENS = [[1], [2, 1, 0], [63, 64, 65], [4095, 4096, 4097, 0, 1], [17, 71, 130, 0, 9000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads,q_len,dtype,lse", [(16, 1, BF16, False), (128, 1, BF16, True), (5, 4, F16, False),
                                                   (64, 2, F16, True), (20, 1, BF16, True), (1, 1, BF16, False),
                                                   (65, 2, BF16, False)])
def test_scores(lens, heads, q_len, dtype, lse):
    run_scores(score_case(lens, heads, q_len, dtype, 64, lse=lse))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("heads,q_len,E,block,unaligned", [(3, 2, 576, 16, 1), (1, 1, 1, 1, 0), (9, 1, 1024, 64, 0), (4, 3, 40, 7, 0),
                                                           (33, 1, 576, 32, 0)])
def test_scores_general(dtype, heads, q_len, E, block, unaligned):
    options = 0 if E != 576 or unaligned or dtype is F32 else GENERAL
    run_scores(score_case([300, 5, 0, 129], heads, q_len, dtype, block, E, lse=True, unaligned=unaligned), options=options)


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scores_of_pages_and_rows(options):
    """Small pages of a long request, an e4m3 cache's scale, padded rows of scores, many requests."""
    run_scores(score_case([20000], 16, 1, F16, 8, scale=0.05), options=options, pad=5)
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 700, 333)
    lens[::6] = 0
    run_scores(score_case(lens.tolist(), 8, 1, BF16, 64), options=options)
    run_scores(score_case([3, 300, 90], 16, 8, BF16, 16), options=options, sm=0.0, pad=1)


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scores_bound_every_entry(options):
    """No entry of a page scores more than the page does."""
    q, cache, table, lens, _ = decode_case([1000, 130, 64], 16, 2, BF16, BF16, 64, nan_tail=False)
    bound = torch.zeros(cache.shape[0], 2, 576, dtype=BF16, device=DEV)
    binding.block_bounds(cache, bound, table, lens)
    score = torch.empty(3, 2, table.shape[1], device=DEV)
    binding.block_scores(q, bound, table, lens, score, block_size=64, sm_scale=0.07, options=options)
    for r, n in enumerate(lens.tolist()):
        kv = cache[table[r, :-(-n // 64)].long()].reshape(-1, 576)[:n].double()
        s = torch.einsum("ihe,ke->ihk", q[r].double(), kv).amax(1) * 0.07
        for c in range(-(-n // 64)):
            # (its own rounding: a few units of 2^-24 of magnitudes below 576 * 16 * 0.07)
            assert (s[:, 64 * c:64 * (c + 1)].amax(1) <= score[r, :, c].double() + 1216 * 2.0 ** -24 * 646).all()


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scores_odd_values(options):
    """NaN of queries and bounds shows; a log sum that is not finite counts as 0; pages outside are -inf."""
    case = score_case([300, 300, 130], 16, 1, BF16, 64, lse=True)
    q, bound, table, lens, block, scale, lse = case
    lse[0, 0, 3], lse[1, 0, 4] = -math.inf, math.nan
    run_scores(case, options=options)
    q[0, 0, 2, 9] = math.nan
    bound[int(table[1, 2]), 1, 100] = math.nan
    q[1, 0, :, 100] = -1.0
    bound[int(table[1, 3]), 0, 7] = math.inf
    q[1, 0, :, 7] = q[1, 0, :, 7].abs() + 1
    table[2, 1] = -1
    out = torch.empty(3, 1, table.shape[1], device=DEV)
    err = i32([0])
    binding.block_scores(q, bound, table, lens, out, block_size=block, sm_scale=0.07, lse=lse, error_flag=err, options=options)
    assert int(err) == binding.FLAG_PHYS_BLOCK
    assert out[0, 0, :5].isnan().all() and out[1, 0, 2].isnan() and out[1, 0, 3] == math.inf
    assert out[1, 0, [0, 1, 4]].isfinite().all() and out[2, 0, 1] == -math.inf and (out[2, 0, 3:] == -math.inf).all()


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scores_lengths_out_of_range(options):
    case = score_case([300, 64, 130], 16, 1, BF16, 64)
    case[3][0], case[3][1] = 10000, -5
    run_scores(case, options=options, flag=binding.FLAG_LENGTH | binding.FLAG_LOGICAL_BLOCK)


# --- select_blocks -----------------------------------------------------------------

def run_select(score, table, lens, block, keep, first, last, flag=0):
    R, n, W = score.shape
    sel, col = (torch.full((R * n, keep), 7, dtype=torch.int32, device=DEV) for _ in range(2))
    sl, err = torch.full((R * n,), 7, dtype=torch.int32, device=DEV), i32([0])
    binding.select_blocks(score, table, lens, sel, sl, block_size=block, first=first, last=last, columns=col, error_flag=err)
    torch.cuda.synchronize()
    assert int(err) == flag
    ids, columns, ln = ref.select(score.tolist(), table.tolist(), lens.tolist(), n, block, keep, first, last)
    assert sel.tolist() == ids and col.tolist() == columns and sl.tolist() == ln
    return sel, sl


@pytest.mark.parametrize("values", ["normal", "few", "equal", "odd"])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 1), (4, 1, 1), (5, 2, 3), (16, 0, 1), (64, 3, 7), (300, 1, 2)])
def test_select(values, keep, first, last):
    lens = [0, 1, 64, 65, 1000, 5003, 33, 20000]
    block, q_len = 64, 3
    table = i32(np.random.default_rng(1).permutation(8 * 320).reshape(8, 320))
    score = normal(gen(keep), 8, q_len, 320)
    if values == "few":
        score = (score * 2).round() / 2
    elif values == "equal":
        score = torch.zeros_like(score)
    elif values == "odd":
        score = (score * 3).round()
        score[:, :, 5::7], score[:, :, 3::11], score[:, :, 2::13], score[:, :, 6::17] = math.nan, math.inf, -math.inf, -0.0
    run_select(score, table, i32(lens), block, keep, first, last)


@pytest.mark.parametrize("width,n,keep", [(20000, 19999, 1000), (9000, 8999, 4500), (8193, 8193, 1), (300, 300, 299), (8192, 8192, 8000)])
def test_select_of_many_pages(width, n, keep):
    """Rows that shared memory does not hold whole; single-token pages."""
    score = (normal(gen(n), 2, 1, width) * 50).round()
    table = torch.arange(2 * width, dtype=torch.int32, device=DEV).view(2, width)
    run_select(score, table, i32([n, n // 3]), 1, keep, 0, 1)


def test_select_strides_and_bad_lengths():
    score = normal(gen(1), 3, 2, 40)[:, :, :30]
    table = torch.arange(90, dtype=torch.int32, device=DEV).view(3, 30)
    table[1, 3] = -5  # passed on
    run_select(score, table, i32([470, -3, 500]), 16, 7, 1, 1, flag=binding.FLAG_LENGTH | binding.FLAG_LOGICAL_BLOCK)
    sel = torch.full((6, 12), 7, dtype=torch.int32, device=DEV)
    sl = i32([0] * 6)
    binding.select_blocks(score, table, i32([470, 100, 480]), sel[:, :7], sl, block_size=16)
    ids, _, ln = ref.select(score.tolist(), table.tolist(), [470, 100, 480], 2, 16, 7, 1, 1)
    assert sel[:, :7].tolist() == ids and (sel[:, 7:] == 7).all() and sl.tolist() == ln


# --- latent_decode_shared --------------------------------------------------------------

def shared_case(members, prefix, lens, heads, q_len, src, cdt, block, dv=512, dr=64, stride=None, seed=8, scale=0.05, gain=1.0):
    rng = np.random.default_rng(seed)
    g = gen(seed)
    both, blocks = mref.tables(rng, list(lens) + list(prefix), block)
    E = dv + dr
    full = normal(g, blocks, block, stride or E)
    full = ((full / scale).clamp(-448, 448) if cdt == FP8 else full).to(cdt)
    for r, n in enumerate(list(lens) + list(prefix)):  # slots past an end hold anything
        if n > 0 and n % block:
            full[int(both[r, n // block]), n % block:] = math.nan
    q = (normal(g, len(lens), q_len, heads, E) * gain).to(src)
    cu = np.concatenate([[0], np.cumsum(members)]) if len(members) else [0]
    return dict(q=q, cache=full[:, :, :E], ptable=i32(both[len(lens):]), plens=i32(prefix), cu=i32(cu),
                table=i32(both[:len(lens)]), lens=i32(lens), scale=torch.tensor([scale], device=DEV) if cdt == FP8 else None,
                dv=dv)


def call_shared(c, out, lse, sm, ws, options=0, err=None, stream=None, q=None):
    binding.latent_decode_shared(c["q"] if q is None else q, c["cache"], c["ptable"], c["plens"], c["cu"], c["table"], c["lens"],
                                 out, lse, sm_scale=sm, scale=c["scale"], workspace=ws, options=options, error_flag=err,
                                 stream=stream)


def new_ws(c):
    return torch.full_like(binding.new_shared_workspace(DEV, *c["q"].shape[:3], c["dv"]), 255)


def run_shared(c, options=0, sm=None, weights_u=None, flag=0, ws=None):
    q = c["q"]
    sm = 1.0 / math.sqrt(192) if sm is None else sm
    out, lse, err = torch.full(q.shape[:3] + (c["dv"],), 7.0, dtype=q.dtype, device=DEV), torch.full(q.shape[:3], 7.0, device=DEV), i32([0])
    call_shared(c, out, lse, sm, new_ws(c) if ws is None else ws, options, err)
    torch.cuda.synchronize()
    assert int(err) == flag
    check_shared(c, out, lse, options, sm, weights_u)
    return out, lse


def check_shared(c, out, lse, options=0, sm=1.0 / math.sqrt(192), weights_u=None):
    q, cache = c["q"], c["cache"]
    f = 1.0 if c["scale"] is None else float(c["scale"])
    want, wl, pv, worst, flat = ref.shared(q, cache, c["ptable"], c["plens"], c["cu"], c["table"], c["lens"], c["dv"], sm, f)
    u, extra, below = mref.U[q.dtype] if weights_u is None else weights_u, 0.0, 0.0
    if cache.dtype == FP8 and options == 0:  # weights and queries in parts, as latent_decode's
        u, below = 2.0 ** -8, 2.0 ** -16 * flat
        extra = sm * 2.0 ** -16.8 * q.double().abs().amax(3) * cache.double().nan_to_num(0).abs().sum(2).max() * f
    mref.check_attention(out, lse, want, wl, pv, worst, q.shape[3], u, extra, below)


@pytest.mark.parametrize("src,cdt", [(BF16, BF16), (F16, F16), (F32, F32), (BF16, FP8), (F16, FP8), (F32, FP8)])
@pytest.mark.parametrize("heads,q_len", [(1, 1), (5, 2), (16, 1)])
def test_shared_general_types(src, cdt, heads, q_len):
    run_shared(shared_case([2, 0, 3], [70, 9, 300], [17, 71, 130, 0, 1, 5], heads, q_len, src, cdt, 16), GENERAL, weights_u=0.0)


@pytest.mark.parametrize("dv,dr,block,stride,heads,q_len", [(512, 64, 1, 577, 3, 1), (40, 8, 7, 48, 9, 3), (1000, 24, 64, 1024, 2, 1),
                                                            (1, 0, 3, 1, 1, 1), (128, 0, 64, 128, 130, 2)])
def test_shared_general_shapes(dv, dr, block, stride, heads, q_len):
    run_shared(shared_case([1, 2], [100, 65], [5, 33, 64], heads, q_len, BF16, BF16, block, dv, dr, stride), 0, weights_u=0.0,
               sm=1 / math.sqrt(dv + dr))


GROUPS = [([1], [1], [1]), ([3], [65], [2, 1, 0]), ([2, 0, 3], [64, 7, 1000], [63, 64, 65, 1, 9]), ([0], [300], [17, 5]),
          ([7], [3000], [0] * 7), ([1, 1, 1, 1], [0, 63, 128, 2000], [17, 71, 130, 0, 3])]


@pytest.mark.parametrize("members,prefix,lens", GROUPS)
@pytest.mark.parametrize("heads,q_len,src,cdt", [(16, 1, BF16, BF16), (128, 1, BF16, BF16), (64, 2, BF16, FP8), (5, 4, F16, F16),
                                                 (20, 1, F16, FP8), (40, 1, BF16, BF16), (1, 1, BF16, FP8), (20, 3, BF16, BF16)])
def test_shared(members, prefix, lens, heads, q_len, src, cdt):
    run_shared(shared_case(members, prefix, lens, heads, q_len, src, cdt, 64))


@pytest.mark.parametrize("block", [8, 16, 24, 48, 128, 200])
@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_shared_page_sizes(block, cdt):
    run_shared(shared_case([3, 2], [700, 65], [block, block + 1, 3, 65, 7], 16, 2, BF16, cdt, block, stride=640))


@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_shared_long_and_many(cdt):
    run_shared(shared_case([4], [20011], [30, 700, 1, 64], 16, 1, BF16, cdt, 64))
    run_shared(shared_case([16, 17], [3001, 5000], [30] * 33, 128, 1, BF16, cdt, 64))
    rng = np.random.default_rng(11)
    members = rng.integers(0, 9, 60)
    run_shared(shared_case(members.tolist(), rng.integers(0, 300, 60).tolist(), rng.integers(0, 90, members.sum() + 3).tolist(), 8, 1,
                           BF16, cdt, 32))


@pytest.mark.parametrize("cdt", [BF16, FP8])
@pytest.mark.parametrize("gain", [12.0, 0.0])
def test_shared_sharp_and_flat(cdt, gain):
    run_shared(shared_case([3, 2], [2500, 100], [400, 3, 64, 900, 1], 16, 1, BF16, cdt, 64, gain=gain))


@pytest.mark.parametrize("options", [0, GENERAL])
def test_shared_bad_data(options):
    c = shared_case([2, 3], [300, 100], [64, 200, 5, 0, 70], 16, 1, BF16, BF16, 64)
    c["ptable"][0, 1], c["table"][1, 0] = -3, c["cache"].shape[0]
    run_shared(c, options, flag=binding.FLAG_PHYS_BLOCK)
    c["plens"][1], c["lens"][2] = 100000, -4
    c["cache"][:] = c["cache"].nan_to_num(0.5)  # (slots behind the ends are seen now)
    run_shared(c, options, flag=binding.FLAG_PHYS_BLOCK | binding.FLAG_LENGTH | binding.FLAG_LOGICAL_BLOCK)


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("cu,flag", [([2, 4, 7], 0), ([0, 3, 100], 0), ([9, 10, 12], 0), ([-2, 3, 7], binding.FLAG_CU_ORDER),
                                     ([5, 2, 5], binding.FLAG_CU_ORDER), ([4, 4, 1], binding.FLAG_CU_ORDER)])
def test_shared_boundaries(options, cu, flag):
    """Boundaries past the requests, requests before and behind the groups, orders that put no request in two groups."""
    c = shared_case([3, 4], [300, 100], [64, 200, 5, 0, 70, 9, 33], 16, 1, BF16, BF16, 64)
    c["cu"] = i32(cu)
    run_shared(c, options, flag=flag)


@pytest.mark.parametrize("options", [0, GENERAL])
def test_shared_without_groups(options):
    c = shared_case([], [], [64, 200, 5], 16, 1, BF16, BF16, 64)
    c["ptable"] = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    out, lse = run_shared(c, options)
    alone, alone_lse = torch.empty_like(out), torch.empty_like(lse)
    binding.latent_decode(c["q"], c["cache"], c["table"], c["lens"], alone, alone_lse, sm_scale=1 / math.sqrt(192), workspace=new_ws(c),
                          options=options)
    assert torch.equal(out, alone) and torch.equal(lse, alone_lse)
    c = shared_case([3], [0], [64, 0, 5], 16, 1, BF16, BF16, 64)
    out, lse = run_shared(c, options)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_shared_strides_stream_graph_and_repeat():
    """Strided q and out, another stream, a captured graph that follows its inputs; the same bits every time."""
    c = shared_case([2, 3], [900, 4000], [900, 17, 400, 1, 64], 16, 2, BF16, BF16, 64)
    want, want_lse = run_shared(c)
    sm = 1 / math.sqrt(192)
    q = torch.zeros(5, 2, 20, 600, dtype=BF16, device=DEV)[:, :, 2:18, 8:584]
    q.copy_(c["q"])
    tall = torch.zeros(2, 5, 16, 576, dtype=BF16, device=DEV).transpose(0, 1)  # tokens of a request far apart
    tall.copy_(c["q"])
    out, lse = torch.zeros(5, 16, 2, 520, dtype=BF16, device=DEV)[:, :, :, 3:515].transpose(1, 2), torch.zeros_like(want_lse)
    side, ws = torch.cuda.Stream(), new_ws(c)
    torch.cuda.synchronize()
    for x in (q, tall):
        out.zero_()
        torch.cuda.synchronize()
        call_shared(c, out, lse, sm, ws, stream=side, q=x)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call_shared(c, out, lse, sm, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    c["plens"].copy_(i32([5, 3999]))
    c["lens"].copy_(i32([2, 0, 399, 1, 64]))
    c["cu"].copy_(i32([1, 3, 5]))
    c["cache"][:] = normal(gen(4), *c["cache"].shape, dtype=BF16)
    graph.replay()
    torch.cuda.synchronize()
    check_shared(c, out, lse)


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("x", [math.nan, math.inf])
def test_shared_odd_values(options, x):
    """NaN and infinities touch the rows that see them: a request's own entries its rows, a prefix's its group's."""
    c = shared_case([2, 2], [300, 20000], [100, 30, 9, 64], 16, 1, BF16, BF16, 64)
    clean, lse0 = run_shared(c, options)
    sm = 1 / math.sqrt(192)
    for place, rows in (((int(c["table"][1, 0]), 5, 570), [1]), ((int(c["ptable"][1, 200]), 7, 3), [2, 3])):
        odd = dict(c, cache=c["cache"].clone())
        odd["cache"][place] = math.nan if x != x else x
        out, lse = torch.empty_like(clean), torch.empty_like(lse0)
        call_shared(odd, out, lse, sm, new_ws(c), options)
        others = [r for r in range(4) if r not in rows]
        assert torch.equal(out[others], clean[others]) and torch.equal(lse[others], lse0[others])
        if x != x:
            assert out[rows].isnan().all() and lse[rows].isnan().all()
    odd = c["q"].clone()
    odd[2, 0, 3, 7] = x
    out, lse = torch.empty_like(clean), torch.empty_like(lse0)
    call_shared(c, out, lse, sm, new_ws(c), options, q=odd)
    assert out[2, 0, 3].isnan().all() and lse[2, 0, 3].isnan()
    out[2, 0, 3], lse[2, 0, 3] = clean[2, 0, 3], lse0[2, 0, 3]
    assert torch.equal(out, clean) and torch.equal(lse, lse0)


# --- together ---------------------------------------------------------------------------

@pytest.mark.parametrize("cdt,heads,q_len", [(BF16, 16, 1), (FP8, 20, 2)])
def test_sparse_step(cdt, heads, q_len):
    """bounds, scores, selection and attention of a step, captured and replayed, against attention over the kept pages."""
    q, cache, table, lens, sc = decode_case([3000, 70, 1, 1500], heads, q_len, BF16, cdt, 64)
    keep, sm, R = 9, 0.07, 4
    bound = torch.zeros(cache.shape[0], 2, 576, dtype=BF16, device=DEV)
    ctx = (lens - q_len).clamp(min=0)
    binding.block_bounds(cache, bound, table, ctx)
    score = torch.empty(R, q_len, table.shape[1], device=DEV)
    sel, sl = torch.empty(R * q_len, keep, dtype=torch.int32, device=DEV), i32([0] * R * q_len)
    out, lse = torch.empty(R * q_len, 1, heads, 512, dtype=BF16, device=DEV), torch.empty(R * q_len, 1, heads, device=DEV)
    ws, err = binding.new_attention_workspace(DEV), i32([0])

    def step():
        binding.block_bounds(cache, bound, table, lens, ctx, err)
        binding.block_scores(q, bound, table, lens, score, block_size=64, sm_scale=sm, scale=sc, error_flag=err)
        binding.select_blocks(score, table, lens, sel, sl, block_size=64, error_flag=err)
        binding.latent_decode(q.view(R * q_len, 1, heads, 576), cache, sel, sl, out, lse, sm_scale=sm, scale=sc, workspace=ws,
                              error_flag=err)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, lse, score, sel, sl):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert int(err) == 0
    f = 1.0 if sc is None else float(sc)
    want, mag = ref.scores(q, bound, table, lens, 64, sm * f)
    fine = want.isfinite()
    assert ((score.double() - want).abs()[fine] <= (1216 + 8) * 2.0 ** -24 * mag[fine]).all()
    ids, _, ln = ref.select(score.tolist(), table.tolist(), lens.tolist(), q_len, 64, keep, 1, 1)
    assert sel.tolist() == ids and sl.tolist() == ln
    from test_mla_ops_gpu import check_decode
    check_decode((q.view(R * q_len, 1, heads, 576), cache, sel, sl, sc), out, lse, sm=sm)

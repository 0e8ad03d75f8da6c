"""Where the operators for long contexts could go wrong besides their sizes: query layouts, far offsets, calls one behind the
other, streams, values that the step before writes."""
import math

import numpy as np
import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import long_reference as ref
import mla_reference as mref
from test_long_ops_gpu import call_shared, check_shared, new_ws, run_scores, run_shared, score_case, shared_case
from test_mla_ops_gpu import BF16, DEV, F16, FP8, GENERAL, decode_case, gen, i32, normal

pytestmark = pytest.mark.gpu
SM = 1 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


@pytest.mark.parametrize("heads,q_len", [(16, 8), (16, 3), (4, 5), (8, 16), (32, 1), (19, 1), (24, 2), (64, 3), (192, 1), (100, 2), (3, 21)])
@pytest.mark.parametrize("layout", ["plain", "padded", "tokens apart"])
def test_shared_query_layouts(heads, q_len, layout):
    """Boxes of new tokens, of requests, of both at one stride, and queries that are none."""
    c = shared_case([5, 3], [700, 70], [64, q_len, 5, 200, 33, 1, 0, 90], heads, q_len, BF16, BF16, 64)
    q = c["q"]
    if layout == "padded":
        c["q"] = torch.zeros(8, q_len + 1, heads + 2, 584, dtype=BF16, device=DEV)[:, :q_len, 1:-1, 8:]
    elif layout == "tokens apart":
        c["q"] = torch.zeros(q_len, 8, heads, 576, dtype=BF16, device=DEV).transpose(0, 1)
    c["q"].copy_(q)
    run_shared(c)


@pytest.mark.parametrize("cdt", [BF16, FP8])
@pytest.mark.parametrize("block", [8, 16, 24, 32, 96])
def test_shared_pairs_page_sizes(cdt, block):
    """Enough rows for pairs of SMs, pages of less than their halves of a tile."""
    run_shared(shared_case([9, 4], [1000, 77], [block, 3, 70, 1, 0, 9, 33, 64, 100, 5, 6, 7, 8], 16, 1, BF16, cdt, block, stride=640))


@pytest.mark.parametrize("src,cdt", [(BF16, BF16), (F16, F16), (BF16, FP8), (F16, FP8)])
@pytest.mark.parametrize("gain", [12.0, 1.0])
def test_shared_pairs_types(src, cdt, gain):
    run_shared(shared_case([20, 1, 0, 40], [3001, 5000, 64, 130], [17] * 64, 16, 1, src, cdt, 64, gain=gain))


@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_shared_growing_scores(cdt):
    """Each tile's scores lie above the last one's, so the running maximum moves at every tile."""
    c = shared_case([12], [1500], [3] * 12, 16, 1, BF16, cdt, 64)
    c["q"][:] = 0.25
    for i in range(24):
        c["cache"][int(c["ptable"][0, i])] = torch.full((64, 576), (i + 1) * 0.125, device=DEV).to(cdt)
    for r in range(12):
        c["cache"][int(c["table"][r, 0])] = torch.full((64, 576), 0.5, device=DEV).to(cdt)
    c["scale"] = None
    run_shared(c, sm=0.2)


@pytest.mark.parametrize("heads,reqs", [(1, 300), (16, 40), (128, 5)])
@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_shared_skewed_groups(heads, reqs, cdt):
    """One request behind a prefix that many shares hold, beside many requests behind short ones."""
    lens = np.random.default_rng(3).integers(0, 40, reqs + 2).tolist()
    run_shared(shared_case([1, reqs, 1], [30000, 50, 9000], lens, heads, 1, BF16, cdt, 64))


@pytest.mark.parametrize("options", [0, GENERAL])
def test_shared_bad_pages_of_pairs(options):
    c = shared_case([9, 4], [1000, 300], [5] * 13, 16, 1, BF16, BF16, 64)
    c["ptable"][0, 2], c["ptable"][0, 15], c["ptable"][1, 0] = -1, c["cache"].shape[0], -7
    run_shared(c, options, flag=binding.FLAG_PHYS_BLOCK)
    c["ptable"][1] = -1  # nothing left of a prefix
    run_shared(c, options, flag=binding.FLAG_PHYS_BLOCK)


@pytest.mark.parametrize("x", [math.nan, math.inf])
def test_shared_odd_values_of_pairs(x):
    for cdt in (BF16, FP8):
        c = shared_case([5, 4], [300, 9000], [9] * 9, 16, 1, BF16, cdt, 64)
        clean, lse0 = run_shared(c)
        odd = c["q"].clone()
        odd[2, 0, 3, 7] = x
        out, lse = torch.empty_like(clean), torch.empty_like(lse0)
        call_shared(c, out, lse, SM, new_ws(c), q=odd)
        assert out[2, 0, 3].isnan().all() and lse[2, 0, 3].isnan()
        out[2, 0, 3], lse[2, 0, 3] = clean[2, 0, 3], lse0[2, 0, 3]
        check_shared(c, out, lse)  # (rows of a CTA may move their references together)
        if x != x:
            spot = dict(c, cache=c["cache"].clone())
            spot["cache"][int(c["ptable"][1, 100]), 7, 3] = math.nan
            call_shared(spot, out, lse, SM, new_ws(c))
            assert out[5:].isnan().all() and lse[5:].isnan().all()
            assert torch.equal(out[:5], clean[:5]) and torch.equal(lse[:5], lse0[:5])


@pytest.mark.parametrize("options", [0, GENERAL])
def test_shared_pages_past_32_bit_offsets(options):
    blocks, block = 120000, 64  # 4.6e9 elements
    cache = torch.empty(blocks, block, 600, dtype=BF16, device=DEV)[:, :, :576]
    pages = [0, blocks - 1, 60001, blocks - 7, 3, blocks - 2]
    for p in pages:
        cache[p] = normal(gen(p + 1), block, 576, dtype=BF16)
    q = normal(gen(9), 6, 1, 16, 576, dtype=BF16)
    c = dict(q=q, cache=cache, ptable=i32([pages[:4]]), plens=i32([230]), cu=i32([0, 6]), table=i32([[pages[4]], [pages[5]]] * 3),
             lens=i32([64, 3, 9, 1, 0, 30]), scale=None, dv=512)
    out, lse = torch.empty(6, 1, 16, 512, dtype=BF16, device=DEV), torch.empty(6, 1, 16, device=DEV)
    call_shared(c, out, lse, 0.07, new_ws(c), options)
    small = dict(c, cache=torch.stack([cache[p] for p in pages]), ptable=i32([[0, 1, 2, 3]]), table=i32([[4], [5]] * 3))
    check_shared(small, out, lse, options, 0.07, None if options == 0 else 0.0)


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scores_of_bounds_past_32_bit_offsets(options):
    blocks = 250000
    bound = torch.empty(blocks, 2, 9600, dtype=BF16, device=DEV)[:, :, :576]  # 4.8e9 elements
    pages = [blocks - 1, 0, 125001, blocks - 9]
    for p in pages:
        bound[p] = normal(gen(p + 1), 2, 576, dtype=BF16)
    q = normal(gen(3), 1, 1, 16, 576, dtype=BF16)
    out = torch.empty(1, 1, 4, device=DEV)
    binding.block_scores(q, bound, i32([pages]), i32([250]), out, block_size=64, sm_scale=0.07, options=options)
    want, mag = ref.scores(q, torch.stack([bound[p] for p in pages]), i32([[0, 1, 2, 3]]), i32([250]), 64, 0.07)
    assert ((out.double() - want).abs() <= (1216 + 8) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("kind", ["small", "pairs", "e4m3", "general"])
def test_shared_calls_one_behind_the_other(kind):
    """The second pass of a call starts before its first one ends, and the next call's first before this one's: calls of
    different inputs in one workspace, and plain decodes between them, without a pause."""
    heads, cdt = {"small": (4, BF16), "pairs": (64, BF16), "e4m3": (64, FP8), "general": (3, BF16)}[kind]
    options = GENERAL if kind == "general" else 0
    cases = [shared_case([3, 2], [900, 70], [64, 17, 400, 1, 64], heads, 1, BF16, cdt, 64, seed=1),
             shared_case([1, 4], [20, 3000], [5, 1000, 40, 0, 9], heads, 1, BF16, cdt, 64, seed=2),
             shared_case([0, 2], [64, 128], [500, 500, 1, 2, 3], heads, 1, BF16, cdt, 64, seed=3)]
    want = [run_shared(c, options, weights_u=0.0 if options else None) for c in cases]
    ws = new_ws(cases[0])
    alone = []
    for c in cases:
        out = torch.empty_like(want[0][0])
        binding.latent_decode(c["q"], c["cache"], c["table"], c["lens"], out, sm_scale=SM, scale=c["scale"], workspace=ws, options=options)
        alone.append(out)
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        c = cases[i * 7 % 3]
        out, lse = torch.full_like(want[0][0], 7.0), torch.full_like(want[0][1], 7.0)
        call_shared(c, out, lse, SM, ws, options)
        between = None
        if i % 4 == 1:
            between = torch.full_like(out, 7.0)
            binding.latent_decode(c["q"], c["cache"], c["table"], c["lens"], between, sm_scale=SM, scale=c["scale"], workspace=ws, options=options)
        got.append((i * 7 % 3, out, lse, between))
    torch.cuda.synchronize()
    for k, out, lse, between in got:
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
        assert between is None or torch.equal(between, alone[k])


def test_shared_on_two_streams():
    """Two calls at once, a workspace each."""
    cases = [shared_case([8, 4], [5000, 700], [64] * 12, 32, 1, BF16, cdt, 64, seed=s) for s, cdt in ((1, BF16), (2, FP8))]
    want = [run_shared(c) for c in cases]
    streams, spaces = [torch.cuda.Stream() for _ in cases], [new_ws(c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = [(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for w in want]
        torch.cuda.synchronize()
        for c, s, ws, (out, lse) in zip(cases, streams, spaces, outs):
            call_shared(c, out, lse, SM, ws, stream=s)
        torch.cuda.synchronize()
        for (out, lse), w in zip(outs, want):
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("cdt,heads", [(BF16, 16), (FP8, 16), (BF16, 128)])
def test_a_step_behind_a_prefix_follows_its_inputs(cdt, heads):
    """plan, append, bounds and shared decode captured once; replays follow the lengths, queries and entries of the moment, which
    the kernels just before write."""
    reqs, block, blocks = 6, 64, 80
    scale = torch.tensor([0.05], device=DEV) if cdt == FP8 else None
    cache = (normal(gen(1), blocks, block, 576) * (20 if cdt == FP8 else 1)).clamp(-448, 448).to(cdt)
    ptable = torch.arange(30, dtype=torch.int32, device=DEV).view(1, 30)
    table = torch.full((reqs, 5), -1, dtype=torch.int32, device=DEV)
    for r in range(reqs):
        table[r, :4] = torch.arange(4, dtype=torch.int32) + 30 + 4 * r
    free = torch.arange(54, 80, dtype=torch.int32, device=DEV)
    ctx, new = i32([0] * reqs), i32([1] * reqs)
    slots = torch.empty(reqs, dtype=torch.int64, device=DEV)
    positions, cu, lens, taken, err = i32([0] * reqs), i32([0] * (reqs + 1)), i32([0] * reqs), i32([0]), i32([0])
    down, q = normal(gen(2), reqs, 576, dtype=BF16), normal(gen(3), reqs, 1, heads, 576, dtype=BF16)
    turn = torch.cat([torch.ones(400, 32, device=DEV), torch.zeros(400, 32, device=DEV)], 1).contiguous()
    bound = torch.zeros(blocks, 2, 576, dtype=BF16, device=DEV)
    plens, groups = i32([1900]), i32([1, 6])
    out, lse = torch.empty(reqs, 1, heads, 512, dtype=BF16, device=DEV), torch.empty(reqs, 1, heads, device=DEV)
    ws = binding.new_shared_workspace(DEV, reqs, 1, heads, 512)

    def step():
        binding.plan_step(ctx, new, table, free, block, slots, positions, None, cu, lens, None, taken, blocks, err)
        binding.append(down[:, :512], down[:, 512:], cache, slots, positions, turn, scale=scale, error_flag=err)
        binding.block_bounds(cache, bound, table, lens, ctx, err)
        binding.latent_decode_shared(q, cache, ptable, plens, groups, table, lens, out, lse, sm_scale=SM, scale=scale, workspace=ws,
                                     error_flag=err)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(4):
        ctx.copy_(i32([(37 * n + 11 * r) % 255 for r in range(reqs)]))
        down.copy_(normal(gen(40 + n), reqs, 576, dtype=BF16))
        q.copy_(normal(gen(50 + n), reqs, 1, heads, 576, dtype=BF16))
        plens.copy_(i32([1900 - 500 * n]))
        before = bound.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err) == 0 and lens.tolist() == [c + 1 for c in ctx.tolist()]
        assert torch.equal(bound, ref.bounds(cache, before, table, lens, ctx))
        check_shared(dict(q=q, cache=cache, ptable=ptable, plens=plens, cu=groups, table=table, lens=lens, scale=scale, dv=512), out, lse)


def test_shared_refuses_a_small_workspace():
    c = shared_case([2], [100], [5, 6], 16, 1, BF16, BF16, 64)
    out = torch.empty(2, 1, 16, 512, dtype=BF16, device=DEV)
    full = new_ws(c)
    for ws, status in ((binding.new_attention_workspace(DEV), 2), (full[:-256], 2), (full[128:], 4)):
        with pytest.raises(binding.PmgError) as e:
            call_shared(c, out, None, SM, ws)
        assert e.value.status == status
    call_shared(c, out, None, SM, full)  # (no log sums)
    check_shared(c, out, run_shared(c)[1])
    with pytest.raises(binding.PmgError):
        binding.shared_workspace_bytes(2, 1, 16, 2000)


def test_calls_of_nothing():
    """No requests, no tokens, no heads, an empty table."""
    i0 = i32([])
    cache, bound = torch.zeros(4, 64, 576, dtype=BF16, device=DEV), torch.zeros(4, 2, 576, dtype=BF16, device=DEV)
    binding.block_bounds(cache, bound, torch.zeros(0, 3, dtype=torch.int32, device=DEV), i0)
    binding.block_bounds(cache, bound, torch.zeros(2, 0, dtype=torch.int32, device=DEV), i32([0, 0]))
    q = torch.zeros(2, 1, 3, 576, dtype=BF16, device=DEV)
    out = torch.full((2, 1, 4), 7.0, device=DEV)
    binding.block_scores(q[:, :, :0], bound, torch.zeros(2, 4, dtype=torch.int32, device=DEV), i32([100, 3]), out, block_size=64, sm_scale=1.0)
    assert (out == -math.inf).all()
    binding.block_scores(q[:0], bound, torch.zeros(0, 4, dtype=torch.int32, device=DEV), i0, out[:0], block_size=64, sm_scale=1.0)
    sel, sl = torch.full((2, 3), 7, dtype=torch.int32, device=DEV), i32([7, 7])
    binding.select_blocks(out[:, :, :0], torch.zeros(2, 0, dtype=torch.int32, device=DEV), i32([0, 0]), sel, sl, block_size=64)
    assert (sel == -1).all() and (sl == 0).all()
    c = shared_case([2], [100], [5, 6], 16, 1, BF16, BF16, 64)
    for empty in (c["q"][:, :0], c["q"][:, :, :0]):
        binding.latent_decode_shared(empty, c["cache"], c["ptable"], c["plens"], c["cu"], c["table"], c["lens"], empty[..., :512],
                                     sm_scale=1.0, workspace=new_ws(c))
    torch.cuda.synchronize()
    c["table"], c["lens"] = torch.zeros(2, 0, dtype=torch.int32, device=DEV), i32([0, 0])  # only a prefix
    run_shared(c)


@pytest.mark.parametrize("heads,q_len", [(200, 1), (128, 3), (96, 2), (130, 2), (1, 130)])
def test_scores_row_chunks(heads, q_len):
    """Rows in several chunks, tokens that end inside one."""
    run_scores(score_case([500, 70, 5000], heads, q_len, BF16, 64, lse=True))


def test_decode_over_selected_pages_is_decode_over_all_where_all_are_kept():
    q, cache, table, lens, sc = decode_case([900, 17, 0, 300], 16, 1, BF16, BF16, 64)
    keep = table.shape[1]
    score = normal(gen(1), 4, 1, keep)
    sel, sl = torch.empty(4, keep, dtype=torch.int32, device=DEV), i32([0] * 4)
    binding.select_blocks(score, table, lens, sel, sl, block_size=64)
    assert torch.equal(sel, torch.where(torch.arange(keep, device=DEV) * 64 < lens[:, None], table, -1)) and torch.equal(sl, lens)
    ws = binding.new_attention_workspace(DEV)
    a, b = (torch.empty(4, 1, 16, 512, dtype=BF16, device=DEV) for _ in range(2))
    binding.latent_decode(q, cache, table, lens, a, sm_scale=SM, workspace=ws)
    binding.latent_decode(q, cache, sel, sl, b, sm_scale=SM, workspace=ws)
    assert torch.equal(a, b)

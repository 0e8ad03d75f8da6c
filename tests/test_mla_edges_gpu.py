"""Where the operators could go wrong besides their sizes: far offsets, many requests, graphs, streams, scales."""
import math

import numpy as np
import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import mla_reference as ref
from test_mla_ops_gpu import BF16, DEV, FP8, GENERAL, check_decode, decode_case, gen, i32, normal, prefill_case, run_append, run_decode, run_prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


@pytest.fixture(scope="module")
def ws():
    return binding.new_attention_workspace(DEV)


@pytest.mark.parametrize("options", [0, GENERAL])
def test_decode_pages_past_32_bit_offsets(ws, options):
    """Pages whose byte and element offsets pass 2^32."""
    blocks, block = 120000, 64  # 4.6e9 elements
    cache = torch.empty(blocks, block, 600, dtype=BF16, device=DEV)[:, :, :576]
    pages = [0, blocks - 1, 60001, blocks - 7]
    for p in pages:
        cache[p] = normal(gen(p + 1), block, 576, dtype=BF16)
    table, lens = i32([pages]), i32([230])
    q = normal(gen(9), 1, 1, 16, 576, dtype=BF16)
    out, lse = torch.empty(1, 1, 16, 512, dtype=BF16, device=DEV), torch.empty(1, 1, 16, device=DEV)
    binding.latent_decode(q, cache, table, lens, out, lse, sm_scale=0.07, workspace=ws, options=options)
    small = torch.stack([cache[p] for p in pages])
    want, wl, pv, worst, _ = ref.decode(q, small, i32([[0, 1, 2, 3]]), lens, 512, 0.07)
    ref.check_attention(out, lse, want, wl, pv, worst, 576, ref.U[BF16])


def test_append_slots_past_32_bit_offsets():
    blocks, block = 120000, 64
    cache = torch.empty(blocks, block, 576, dtype=BF16, device=DEV)
    c, kp = normal(gen(1), 3, 512, dtype=BF16), normal(gen(2), 3, 64, dtype=BF16)
    slots = torch.tensor([blocks * block - 1, 5, 70000 * block + 3], device=DEV)
    cs = torch.cat([torch.ones(4, 32, device=DEV), torch.zeros(4, 32, device=DEV)], 1).contiguous()
    binding.append(c, kp, cache, slots, i32([0, 1, 2]), cs)
    got = cache.view(-1, 576)[slots]
    assert torch.equal(got, torch.cat([c, kp], 1))


@pytest.mark.parametrize("options", [0, GENERAL])
def test_prefill_rows_past_32_bit_offsets(ws, options):
    tk, heads = 72000, 128  # 2.36e9 elements
    kv = torch.empty(tk, heads, 256, dtype=BF16, device=DEV)
    kv[-200:] = normal(gen(3), 200, heads, 256, dtype=BF16)
    pe = torch.empty(tk, 64, dtype=BF16, device=DEV)
    pe[-200:] = normal(gen(4), 200, 64, dtype=BF16)
    q = normal(gen(5), 70, heads, 192, dtype=BF16)
    out, lse = torch.empty(70, heads, 128, dtype=BF16, device=DEV), torch.empty(70, heads, device=DEV)
    cu_q, cu_k = i32([0, 0, 70]), i32([0, tk - 200, tk])
    binding.latent_prefill(q, kv[:, :, :128], pe, kv[:, :, 128:], cu_q, cu_k, out, lse, sm_scale=0.07, causal=True,
                           workspace=ws, options=options)
    want, wl, pv, worst = ref.prefill(q, kv[-200:, :, :128], pe[-200:], kv[-200:, :, 128:], [0, 70], [0, 200], 0.07, True)
    ref.check_attention(out, lse, want, wl, pv, worst, 192, ref.U[BF16])


@pytest.mark.parametrize("reqs", [32, 33, 500])
@pytest.mark.parametrize("options", [0, GENERAL])
def test_many_requests(ws, reqs, options):
    rng = np.random.default_rng(reqs)
    lens = rng.integers(0, 90, reqs)
    lens[::7] = 0
    run_decode(decode_case(lens.tolist(), 8, 1, BF16, BF16, 16), ws, options=options)
    q_lens = np.minimum(rng.integers(0, 40, reqs), lens)
    for causal in (False, True):
        run_prefill(prefill_case(q_lens.tolist(), lens.tolist(), 2, BF16, prev=True), ws, causal, options)


@pytest.mark.parametrize("options", [0, GENERAL])
def test_scale_of_zero(ws, options):
    """Every seen key weighs the same."""
    run_decode(decode_case([100, 7], 16, 2, BF16, BF16, 16), ws, options=options, sm=0.0)
    run_decode(decode_case([100, 7], 16, 2, BF16, FP8, 16), ws, options=options, sm=0.0)
    run_prefill(prefill_case([30, 5], [130, 5], 2, BF16), ws, True, options, sm=0.0)


def test_rows_that_see_nothing(ws):
    """More new tokens than entries: the first rows see none; a prefill of more queries than keys likewise."""
    for options in (0, GENERAL):
        for cdt in (BF16, FP8):
            out, lse = run_decode(decode_case([2, 5, 0], 16, 4, BF16, cdt, 16), ws, options=options)
            assert (out[0, :2] == 0).all() and (lse[0, :2] == -math.inf).all() and (lse[0, 2:] > -math.inf).all()
        out, lse = run_prefill(prefill_case([300, 200], [50, 0], 2, BF16), ws, True, options)
        assert (out[:250] == 0).all() and (lse[:250] == -math.inf).all() and (lse[250:300] > -math.inf).all()


def test_entries_that_share_pages(ws):
    """Requests with a common prefix name the same pages."""
    q, cache, table, lens, sc = decode_case([300, 300, 300], 16, 1, BF16, BF16, 64, nan_tail=False)
    table[1, :3], table[2, :4] = table[0, :3], table[0, :4]
    run_decode((q, cache, table, lens, sc), ws)


def test_a_step_in_a_graph_follows_its_inputs(ws):
    """plan, append and decode captured once; replays follow the lengths, queries and entries of the moment."""
    reqs, heads, block = 3, 16, 16
    ctx, new = i32([20, 0, 100]), i32([1, 1, 1])
    table = torch.full((reqs, 16), -1, dtype=torch.int32, device=DEV)
    for r in range(reqs):
        table[r, :8] = torch.arange(8, dtype=torch.int32) + 8 * r
    free = torch.arange(24, 40, dtype=torch.int32, device=DEV)
    cache = normal(gen(1), 40, block, 576, dtype=BF16)
    slots = torch.empty(4, dtype=torch.int64, device=DEV)
    positions, t2s, cu, cu_seq = i32([0] * 4), i32([0] * 4), i32([0] * 4), i32([0] * 4)
    lens, taken = i32([0] * 3), i32([0])
    down, q = normal(gen(2), 4, 576, dtype=BF16), normal(gen(3), 4, heads, 576, dtype=BF16)
    cs = torch.cat([torch.ones(200, 32, device=DEV), torch.zeros(200, 32, device=DEV)], 1).contiguous()
    out = torch.empty(reqs, 1, heads, 512, dtype=BF16, device=DEV)

    def step():
        binding.plan_step(ctx, new, table, free, block, slots, positions, t2s, cu, lens, cu_seq, taken, 40)
        binding.append(down[:, :512], down[:, 512:], cache, slots, positions, cs, q_pe=q[:, :, 512:], q_out=q[:, :, 512:])
        binding.latent_decode(q[:3].view(3, 1, heads, 576), cache, table, lens, out, sm_scale=0.07, workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lengths in ([20, 0, 100], [31, 15, 127], [32, 16, 5]):
        ctx.copy_(i32(lengths))
        down.copy_(normal(gen(sum(lengths)), 4, 576, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [n + 1 for n in lengths]
        assert slots.tolist()[:3] == [int(table[r, n // block]) * block + n % block for r, n in enumerate(lengths)]
        assert slots[3] == -1 and positions[3] == -1
        for r, n in enumerate(lengths):
            assert torch.equal(cache[int(table[r, n // block]), n % block], down[r])
        want, _, pv, worst, _ = ref.decode(q[:3].view(3, 1, heads, 576), cache, table, lens, 512, 0.07)
        err = (out.double() - want).abs()
        assert (err <= ref.U[BF16] * want.abs() + (ref.U[BF16] + 1e-3) * pv).all()


def test_prefill_on_another_stream_and_in_a_graph(ws):
    c = prefill_case([300, 77], [900, 500], 4, BF16)
    want, _ = run_prefill(c, ws, True)
    out, side, ws2 = torch.zeros_like(want), torch.cuda.Stream(), torch.empty_like(ws).fill_(255)
    torch.cuda.synchronize()
    args = (c["q"], c["k"], c["pe"], c["v"], c["cu_q"], c["cu_k"], out)
    kw = dict(sm_scale=1 / math.sqrt(192), causal=True, workspace=ws2)
    binding.latent_prefill(*args, **kw, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.latent_prefill(*args, **kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("cdt", [BF16, FP8])
@pytest.mark.parametrize("n,block", [(300, 64), (300, 16), (20000, 64)])
def test_decode_odd_values_in_unseen_entries(ws, options, cdt, n, block):
    """A row of an earlier token does not meet the infinities and NaN of a later token's entry; a row that sees them has NaN."""
    q, cache, table, lens, sc = decode_case([n, 90], 16, 4, BF16, cdt, block)
    clean, lse0 = run_decode((q, cache, table, lens, sc), ws, options=options)
    places = [(n - 1, 5), (n - 2, 570), (n - 1, 400)]
    odd = cache.clone()
    for i, (j, d) in enumerate(places):
        odd[int(table[0, j // block]), j % block, d] = math.nan if cdt is FP8 or i < 2 else math.inf
    out, lse = torch.empty_like(clean), torch.empty(2, 4, 16, device=DEV)
    binding.latent_decode(q, odd, table, lens, out, lse, sm_scale=1 / math.sqrt(192), scale=sc, workspace=ws, options=options)
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all() and lse[0, :2].isfinite().all()
    out[0, 2:], lse[0, 2:] = clean[0, 2:], lse0[0, 2:]
    check_decode((q, cache, table, lens, sc), out, lse, options=options)


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("q_len,k_len", [(300, 300), (300, 700), (130, 9000), (40, 20)])
def test_prefill_odd_values_in_unseen_keys(ws, options, dtype, q_len, k_len):
    """Only rows that see a key have its infinities and NaN, and those only in their columns."""
    c = prefill_case([q_len, 50], [k_len, 50], 3, dtype)
    clean, lse0 = run_prefill(c, ws, True, options)
    v = c["v"].clone()
    places = [(k_len - 1, 0, 5, math.nan), (k_len - 17, 1, 127, math.inf), (k_len - 18, 1, 64, -math.inf),
              (max(k_len - 130, 0), 2, 0, math.nan)]
    want = clean.clone()
    rows = torch.arange(q_len, device=DEV)
    for j, h, d, x in places:
        v[j, h, d] = x
        sees = rows + k_len - q_len >= j
        want[:q_len, h, d] = torch.where(sees, torch.tensor(x, dtype=dtype, device=DEV), want[:q_len, h, d])
    out, lse = torch.empty_like(clean), torch.empty_like(lse0)
    binding.latent_prefill(c["q"], c["k"], c["pe"], v, c["cu_q"], c["cu_k"], out, lse, sm_scale=1 / math.sqrt(192),
                           causal=True, workspace=ws, options=options)
    assert torch.equal(lse, lse0)
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("x", [math.nan, math.inf])
@pytest.mark.parametrize("n", [100, 20000])
def test_odd_queries_make_their_row_nan(ws, options, x, n):
    """Result and log sum, whether one share holds the row or several; other rows do not change."""
    for src, cdt in ((BF16, BF16), (BF16, FP8), (torch.float16, FP8)):
        q, cache, table, lens, sc = decode_case([n], 16, 1, src, cdt, 64)
        clean, lse0 = run_decode((q, cache, table, lens, sc), ws, options=options)
        out, lse = torch.empty_like(clean), torch.empty_like(lse0)
        odd = q.clone()
        odd[0, 0, 3, 7] = x
        binding.latent_decode(odd, cache, table, lens, out, lse, sm_scale=1 / math.sqrt(192), scale=sc, workspace=ws,
                              options=options)
        assert out[0, 0, 3].isnan().all() and lse[0, 0, 3].isnan()
        out[0, 0, 3], lse[0, 0, 3] = clean[0, 0, 3], lse0[0, 0, 3]
        check_decode((q, cache, table, lens, sc), out, lse, options=options)
    c = prefill_case([130], [n + 130], 2, BF16)
    clean, lse0 = run_prefill(c, ws, True, options)
    want, wl, pv, worst = ref.prefill(c["q"], c["k"], c["pe"], c["v"], c["cu_q"], c["cu_k"], 1 / math.sqrt(192), True)
    odd = c["q"].clone()
    odd[77, 1, 7] = x
    out, lse = torch.empty_like(clean), torch.empty_like(lse0)
    binding.latent_prefill(odd, c["k"], c["pe"], c["v"], c["cu_q"], c["cu_k"], out, lse, sm_scale=1 / math.sqrt(192),
                           causal=True, workspace=ws, options=options)
    assert out[77, 1].isnan().all() and lse[77, 1].isnan()
    out[77, 1], lse[77, 1] = clean[77, 1], lse0[77, 1]
    ref.check_attention(out, lse, want, wl, pv, worst, 192, ref.U[BF16])


@pytest.mark.parametrize("t,dr,heads,src,unaligned,inplace", [
    (2100, 64, 65, BF16, 0, False), (8192, 64, 16, BF16, 0, True), (2100, 64, 33, torch.float32, 0, False),
    (700, 256, 49, torch.float16, 0, False), (9001, 8, 130, torch.float16, 0, True), (66000, 128, 1, BF16, 0, False),
    (2100, 64, 65, BF16, 3, False)])
@pytest.mark.parametrize("pairs", [True, False])
def test_append_large(t, dr, heads, src, unaligned, inplace, pairs):
    """Calls whose queries are launched by themselves."""
    assert t * heads * dr * (4 if src is torch.float32 else 2) >= 2 ** 24
    run_append(t, 64, dr, heads, src, FP8 if heads % 2 else src, 64, 64 + dr, pairs, unaligned=unaligned, inplace=inplace)


def test_append_large_skips_tokens_and_repeats():
    t, heads, dr = 9000, 16, 64
    g = gen(4)
    c, kp, q = normal(g, t, 64, dtype=BF16), normal(g, t, dr, dtype=BF16), normal(g, t, heads, dr, dtype=BF16)
    cs = torch.rand(500, dr, generator=g, device=DEV)
    positions = torch.as_tensor(np.random.default_rng(1).integers(0, 500, t).astype(np.int32), device=DEV)
    positions[::7], positions[5], positions[8990:] = -1, 500, -1
    slots = torch.where((positions >= 0) & (positions < 500), torch.arange(t, device=DEV), -1)
    cache = torch.zeros(150, 64, 128, dtype=BF16, device=DEV)
    want = None
    for _ in range(3):
        out, err = torch.full_like(q, 7.0), i32([0])
        binding.append(c, kp, cache, slots, positions, cs, q_pe=q, q_out=out, error_flag=err)
        got = out.clone()  # follows in the stream
        assert int(err) == binding.FLAG_POSITION
        skipped = slots < 0
        assert (got[skipped] == 7).all()
        turned, mag = ref.rotate(q[~skipped].double(), cs.double()[positions[~skipped].long()], False)
        assert ((got[~skipped].double() - turned).abs() <= ref.U[BF16] * turned.abs() + mag * 2.0 ** -21).all()
        want = got if want is None else want
        assert torch.equal(got, want) and torch.equal(cache.view(-1, 128)[slots[~skipped], :64], c[~skipped])

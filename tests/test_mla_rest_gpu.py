"""Latent attention where neighbours, leftovers and limits could reach a result: what is in shared memory before a call,
and lengths next to the largest."""
import math

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

from test_mla_ops_gpu import BF16, DEV, F16, FP8, check_decode, decode_case, gen, i32, normal, run_decode

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


@pytest.mark.parametrize("cdt", [BF16, FP8])
@pytest.mark.parametrize("q_len,short", [(1, 0), (3, 1), (2, 63), (2, 64)])
def test_decode_of_the_longest_request(ws, cdt, q_len, short):
    """INT32_MAX entries and a few fewer, of which the table holds the last page: the others' are left out."""
    block, heads = 4096, 16
    longest = 2 ** 31 - 1 - short
    q, cache, _, _, sc = decode_case([block, 70], heads, q_len, BF16, cdt, block, nan_tail=False)
    table = torch.full((2, 2 ** 31 // block), -1, dtype=torch.int32, device=DEV)
    table[0, -1], table[1, 0] = 1, 0
    out, lse = torch.empty(2, q_len, heads, 512, dtype=BF16, device=DEV), torch.empty(2, q_len, heads, device=DEV)
    err = i32([0])
    binding.latent_decode(q, cache, table, i32([longest, 70]), out, lse, sm_scale=SM, scale=sc, workspace=ws, error_flag=err)
    torch.cuda.synchronize()
    assert int(err) == binding.FLAG_PHYS_BLOCK
    few = i32([[1], [0]])
    check_decode((q, cache, few, i32([longest % block, 70]), sc), out, lse)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("few", [0, 127, 128])
def test_prefill_over_the_most_keys(ws, causal, few):
    """INT32_MAX keys and a few fewer: rows that overlap, all 0 but the end of the last one, which weighs as much as all
    others together."""
    tk, tq = 2 ** 31 - 1 - few, 3
    flat = torch.zeros(8 * (tk - 1) + 128, dtype=BF16, device=DEV)
    flat[-8] = 1.0
    rows = flat.as_strided((tk, 1, 128), (8, 128, 1))
    q = torch.zeros(tq, 1, 192, dtype=BF16, device=DEV)
    q[:, :, 120] = math.log(tk) / SM
    out, lse = torch.empty(tq, 1, 128, dtype=BF16, device=DEV), torch.empty(tq, 1, device=DEV)
    binding.latent_prefill(q, rows, flat.as_strided((tk, 64), (8, 1)), rows, i32([0, tq]), i32([0, tk]), out, lse,
                           sm_scale=SM, causal=causal, workspace=ws)
    # the last key's weight in 64 bits; other rows of keys and values meet that element nowhere
    strong = math.exp(float(q[0, 0, 120].double()) * SM)
    for i in range(tq):
        sees = tk - (tq - 1 - i if causal else 0)
        others, w = (tk - 1, strong) if sees == tk else (sees, 0.0)
        # sums of 1 are exact up to 2^24 in a share and joined in 32 bits; the score is one product, its weight's error 2^-19
        assert abs(float(lse[i, 0]) - math.log(others + w)) < 2.0 ** -18 * 22
        got = out[i, 0].double()
        assert abs(float(got[120]) - w / (others + w)) <= 2.0 ** -8 + 2.0 ** -16
        got[120] = 0.0
        assert (got == 0).all()


def test_plan_takes_neighbours_in_one_buffer():
    """Inputs and results side by side in one tensor do not overlap."""
    r, n = 3, 9
    buffer = torch.full((53,), 7, dtype=torch.int32, device=DEV)
    cut = iter(buffer.split([r, r, 4, 4 * r, r, r + 1, r + 1, 1, 1, n, n]))
    ctx, new, free, table, lens, cu, cu_seq, taken, err, positions, t2s = (next(cut) for _ in range(11))
    ctx.copy_(i32([3, 0, 4]))
    new.copy_(i32([2, 4, 1]))
    free.copy_(i32([9, 8, 7, 6]))
    table.copy_(i32([0, -1, -1, -1, -1, -1, -1, -1, 1, -1, -1, -1]))
    err.zero_()
    slots = torch.empty(n, dtype=torch.int64, device=DEV)
    binding.plan_step(ctx, new, table.view(r, 4), free, 4, slots, positions, t2s, cu, lens, cu_seq, taken, 10, err)
    assert table.tolist() == [0, 9, -1, -1, 8, -1, -1, -1, 1, 7, -1, -1] and int(taken) == 3 and int(err) == 0
    assert slots.tolist() == [3, 36, 32, 33, 34, 35, 28, -1, -1] and positions.tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert t2s.tolist() == [0, 0, 1, 1, 1, 1, 2, -1, -1]
    assert lens.tolist() == [5, 4, 5] and cu.tolist() == [0, 2, 6, 7] and cu_seq.tolist() == [0, 5, 9, 14]
    assert ctx.tolist() == [3, 0, 4] and new.tolist() == [2, 4, 1] and free.tolist() == [9, 8, 7, 6]

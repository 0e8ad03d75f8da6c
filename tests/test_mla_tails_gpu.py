"""One strong key beside a long tail of weak ones: what the tail adds up to must arrive, however small each weight is.

Queries and entries are chosen so that everything but the weights is exact: e4m3 entries are given as such, queries as
their parts hold them, the strong key is the request's first entry and its value is 0, the others' values have a common
mean. So the result is the tail's share alone, and a bound that is relative to it has no room for weights that vanish.

Weights of an e4m3 cache are held as fp16 in three e5m2 parts: to 2^-11 and 2^-9 of their value, or, where that is more, to
half a step of 2^-28 of the largest weight, which is at most 2^-8.7 of a tail's usual weight here: together below 2^-8.
Weights of 16-bit products have their type's rounding: 2^-8, or 2^-11 with the subnormal ones' half step far below it."""
import math

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import mla_reference as ref
from test_mla_ops_gpu import BF16, DEV, F16, FP8, GENERAL, gen, i32, normal

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


def four_bits(x):
    """Values of at most four significant bits near x."""
    return x.to(FP8).float()


def tail_case(lens, heads, q_len, src, cdt, octaves, spread, block=64, scale=0.0625, seed=5):
    """Requests whose first entry has 2^octaves times the weight of a usual one; `spread`: of the others' scores, in nats."""
    g = gen(seed)
    pages = [-(-n // block) for n in lens]
    blocks = sum(pages)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    entry = torch.cat([1.0 + 0.5 * normal(g, blocks, block, 512), normal(g, blocks, block, 64)], 2)
    entry[:, :, 512] = 0.0  # the strong key's own value
    f = scale if cdt is FP8 else 1.0
    entry = four_bits(entry / f)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
        first = entry[int(table[r, 0]), 0]
        first.zero_()
        first[512] = 16.0 / f
    # q . e = sum over 63 rotated values of standard deviation `spread` / SM, and what raises the first
    q = torch.zeros(len(lens), q_len, heads, 576, device=DEV)
    q[..., 513:] = four_bits(normal(g, len(lens), q_len, heads, 63).sign() * spread / SM / math.sqrt(63))
    q[..., 512] = octaves * math.log(2) / SM / 16.0
    return q.to(src), entry.to(cdt), table, i32(lens), (torch.tensor([scale], device=DEV) if cdt is FP8 else None)


def run_tail(ws, case, weights_u, options=0):
    q, cache, table, lens, sc = case
    out = torch.full(q.shape[:3] + (512,), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    err = i32([0])
    binding.latent_decode(q, cache, table, lens, out, lse, sm_scale=SM, scale=sc, workspace=ws, error_flag=err,
                          options=options)
    torch.cuda.synchronize()
    assert int(err) == 0
    want, wl, pv, worst, _ = ref.decode(q, cache, table, lens, 512, SM, 1.0 if sc is None else float(sc))
    assert (want.abs() > 1e-6).any()
    ref.check_attention(out, lse, want, wl, pv, worst, 576, weights_u)


def strong(n, share):
    """Octaves that give the first of n keys this share: the others' mean weight is e^(1/2) of their usual one."""
    return math.log2(share / (1 - share) * n * math.exp(0.5))


@pytest.mark.parametrize("src", [BF16, F16])
@pytest.mark.parametrize("share", [0.3, 0.5, 0.9])
@pytest.mark.parametrize("heads,q_len,lens", [
    (128, 40, [16384]),            # so many rows that a unit has the whole request
    (16, 1, [16384]),              # cut into many shares
    (64, 2, [16384, 700, 9000]),
    (20, 1, [4096] * 160)])        # a request or so a unit
def test_decode_fp8_tail(ws, src, share, heads, q_len, lens):
    run_tail(ws, tail_case(lens, heads, q_len, src, FP8, strong(max(lens), share), 1.0), 2.0 ** -8)


@pytest.mark.parametrize("src", [BF16, F16])
@pytest.mark.parametrize("octaves", [6.3, 11.4, 16.7, 19.3])
def test_decode_fp8_even_tail(ws, src, octaves):
    """Every key of the tail has the same weight, so its rounding does not average out."""
    run_tail(ws, tail_case([8000, 64, 65], 32, 1, src, FP8, octaves, 0.0), 2.0 ** -8)
    run_tail(ws, tail_case([3000] * 100, 128, 1, src, FP8, octaves, 0.0), 2.0 ** -8)


@pytest.mark.parametrize("options", [0, GENERAL])
@pytest.mark.parametrize("src", [BF16, F16])
def test_decode_tail(ws, src, options):
    """16-bit caches; for fp16, weights that are subnormal where the largest is 1."""
    for octaves in (6.3, 14.6, 20.5):
        u = ref.U[src] if options == 0 else 0.0
        run_tail(ws, tail_case([8000, 64, 65], 32, 1, src, src, octaves, 0.0), u, options)
        run_tail(ws, tail_case([1000] * 100, 128, 1, src, src, octaves, 0.0), u, options)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("octaves", [6.3, 14.6, 20.5])
def test_prefill_tail(ws, dtype, causal, octaves):
    g = gen(7)
    heads, lq, lk = 128, 300, 2000  # more row tiles than SMs: most shares hold whole ones
    kv = torch.cat([torch.zeros(lk, heads, 128, device=DEV), 1.0 + 0.5 * normal(g, lk, heads, 128)], 2)
    kv[0] = 0.0
    pe = torch.zeros(lk, 64, device=DEV)
    pe[0, 0] = 16.0
    q = torch.zeros(lq, heads, 192, device=DEV)
    q[:, :, 128] = octaves * math.log(2) / SM / 16.0
    kv, pe, q = kv.to(dtype), pe.to(dtype), q.to(dtype)
    cu_q, cu_k = i32([0, lq]), i32([0, lk])
    out, lse = torch.empty(lq, heads, 128, dtype=dtype, device=DEV), torch.empty(lq, heads, device=DEV)
    binding.latent_prefill(q, kv[:, :, :128], pe, kv[:, :, 128:], cu_q, cu_k, out, lse, sm_scale=SM, causal=causal,
                           workspace=ws)
    want, wl, pv, worst = ref.prefill(q, kv[:, :, :128], pe, kv[:, :, 128:], [0, lq], [0, lk], SM, causal)
    ref.check_attention(out, lse, want, wl, pv, worst, 192, ref.U[dtype])

"""The operators around the gather on the GPU against their 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

import mla_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16, F32, FP8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


@pytest.fixture(scope="module")
def ws():
    return binding.new_attention_workspace(DEV)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


# --- plan_step -------------------------------------------------------------------

def run_plan(ctx, new, table, free, block, num_blocks, max_tokens):
    r = len(ctx)
    o = dict(slots=torch.full((max_tokens,), 7, dtype=torch.int64, device=DEV),
             positions=torch.full((max_tokens,), 7, dtype=torch.int32, device=DEV),
             t2s=torch.full((max_tokens,), 7, dtype=torch.int32, device=DEV), cu_new=i32([7] * (r + 1)),
             lens=i32([7] * r), cu_seq=i32([7] * (r + 1)), taken=i32([7]), err=i32([0]))
    bt = i32(table).view(r, -1)
    binding.plan_step(i32(ctx), i32(new), bt, i32(free), block, o["slots"], o["positions"], o["t2s"], o["cu_new"],
                      o["lens"], o["cu_seq"], o["taken"], num_blocks, o["err"])
    torch.cuda.synchronize()
    return ([bt.tolist()] + [o[k].tolist() for k in ("slots", "positions", "t2s", "cu_new", "lens", "cu_seq")]
            + [int(o["taken"])], int(o["err"]))


@pytest.mark.parametrize("reqs,ctx_hi,new_hi,block,pad", [
    (1, 0, 1, 64, 0), (1, 100, 300, 7, 5), (4, 70, 1, 64, 0), (64, 3000, 1, 64, 17), (33, 40, 90, 16, 0),
    (513, 100, 40, 1, 0), (4096, 30, 9, 16, 3), (4097, 30, 9, 16, 0), (9000, 8, 5, 3, 1000), (5, 0, 0, 16, 4)])
def test_plan_matches_definition(reqs, ctx_hi, new_hi, block, pad):
    rng = np.random.default_rng(reqs * 7 + block)
    ctx, new = rng.integers(0, ctx_hi + 1, reqs), rng.integers(0, new_hi + 1, reqs)
    table, used = ref.tables(rng, ctx.tolist(), block, spare=0)
    need = int((-(-(ctx + new) // block) - -(-ctx // block)).sum())
    width = int(max(1, (-(-(ctx + new) // block)).max()))
    wide = np.full((reqs, width), -1, np.int32)
    wide[:, :min(width, table.shape[1])] = table[:, :width]
    free = used + rng.permutation(need + 2)
    tokens = int(new.sum()) + pad
    got, err = run_plan(ctx, new, wide, free, block, used + need + 2, tokens)
    assert err == 0
    want = ref.plan(ctx, new, wide, free, block, used + need + 2, tokens)
    for g, w in zip(got, want):
        assert g == w


def test_plan_bad_data():
    # request 0 runs out of its row, 1 has a bad cached page, 2 a negative length, 3 finds no free block
    ctx, new = [6, 6, -5, 0, 3], [9, 1, 2, 6, 1]
    table = [[0, 1, -1], [2, 99, -1], [-1, -1, -1], [-1, -1, -1], [3, -1, -1]]
    free = [5, 77, 6, 7]  # 77 is no block; request 0 takes pages 2 and 3
    got, err = run_plan(ctx, new, table, free, 4, 10, 19)
    want = ref.plan(ctx, new, table, free, 4, 10, 19)
    assert got == list(want)
    assert err == (binding.FLAG_LOGICAL_BLOCK | binding.FLAG_PHYS_BLOCK | binding.FLAG_LENGTH | binding.FLAG_NO_BLOCKS)
    # fewer rows than tokens: the rest is dropped
    got, err = run_plan([0], [9], [[-1]], [0], 16, 1, 5)
    assert got[1] == [0, 1, 2, 3, 4] and err == binding.FLAG_CAPACITY


def test_plan_of_no_requests():
    slots = torch.full((3,), 7, dtype=torch.int64, device=DEV)
    cu = i32([7])
    empty = i32([])
    binding.plan_step(empty, empty, torch.zeros(0, 4, dtype=torch.int32, device=DEV), empty, 16, slots, None, None, cu,
                      empty, None, None, 5)
    assert slots.tolist() == [-1] * 3 and cu.tolist() == [0]


# --- append ----------------------------------------------------------------------

def run_append(t, dv, dr, heads, src, cdt, block, stride, pairs, norm=True, unaligned=0, seed=1, scale=0.05, inplace=False):
    g = gen(seed)
    rng = np.random.default_rng(seed)
    down = normal(g, t, dv + dr + unaligned, dtype=src)
    c, kp = down[:, unaligned:unaligned + dv], down[:, unaligned + dv:]
    w = 1 + 0.1 * normal(g, dv) if norm else None
    positions = torch.as_tensor(rng.integers(0, 500, t).astype(np.int32), device=DEV)
    angle = torch.rand(500, dr // 2, generator=g, device=DEV) * 6.28
    cs = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
    blocks = -(-t // block) + 2
    full = torch.zeros(blocks, block, stride, device=DEV).to(cdt)
    full.view(torch.uint8).fill_(0x21)
    before = full.clone()
    cache = full[:, :, :dv + dr]
    slots = torch.as_tensor(rng.permutation(blocks * block)[:t].astype(np.int64), device=DEV)
    slots[t // 2::5] = -1  # padding
    sc = torch.tensor([scale], device=DEV) if cdt == FP8 else None
    q = normal(g, t, heads, dr + 3 * (unaligned > 0), dtype=src)[:, :, -dr:] if heads else None
    qo = (q if inplace else torch.zeros(t, heads, dv + dr, dtype=src, device=DEV)[:, :, dv:]) if heads else None
    q0 = q.double() if heads else None
    err = i32([0])
    binding.append(c, kp, cache, slots, positions, cs, norm_weight=w, eps=1e-6, scale=sc, q_pe=q, q_out=qo,
                   interleaved=pairs, error_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    x = c.double()
    latent = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double() if norm else x
    turn, mag = ref.rotate(kp.double(), cs.double()[positions.long()], pairs)
    f = float(sc) if sc is not None else 1.0
    want = torch.cat([latent, turn], 1) / f
    # 32 bits: the mean's sum and square root (dv + 8 roundings at most, of positive terms), three products; a rotation
    slack = torch.cat([latent.abs() * (dv + 16) * 2.0 ** -24, mag * 4 * 2.0 ** -24], 1) / f
    if cdt == FP8:
        want = want.clamp(-448, 448)
    real = slots >= 0
    block_of, at = slots[real] // block, slots[real] % block
    got = cache[block_of, at].double()
    tiny = {FP8: 2.0 ** -10, F16: 2.0 ** -25}.get(cdt, 0.0)  # half a step among the subnormal values
    bound = ref.U[cdt] * want[real].abs() + slack[real] * 1.1 + tiny
    assert ((got - want[real]).abs() <= bound).all()
    # nothing else is written
    mask = torch.zeros(blocks * block, dtype=torch.bool, device=DEV)
    mask[slots[real]] = True
    same = full.view(torch.uint8).view(blocks * block, -1) == before.view(torch.uint8).view(blocks * block, -1)
    assert same[~mask].all()
    assert same.view(blocks * block, stride, -1)[:, dv + dr:].all()
    if heads:
        wq, mq = ref.rotate(q0, cs.double()[positions.long()], pairs)
        tiny = 2.0 ** -25 if src == F16 else 0.0
        assert ((qo.double() - wq).abs() <= ref.U[src] * wq.abs() + mq * 4.4 * 2.0 ** -24 + tiny).all()


@pytest.mark.parametrize("src,cdt", [(BF16, BF16), (BF16, FP8), (F16, F16), (F16, FP8), (F32, F32), (F32, FP8),
                                     (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("pairs", [True, False])
def test_append_types(src, cdt, pairs):
    run_append(37, 512, 64, 5, src, cdt, 16, 640, pairs)


@pytest.mark.parametrize("t,dv,dr,heads,block,stride,unaligned,norm,inplace", [
    (1, 512, 64, 16, 64, 576, 0, True, False), (1, 512, 64, 0, 64, 576, 0, True, False),
    (300, 512, 64, 128, 64, 576, 0, True, True), (65, 512, 64, 17, 1, 577, 0, True, False),
    (65, 512, 64, 17, 48, 576, 3, False, True), (9, 8, 2, 3, 5, 10, 0, True, False), (9, 1024, 128, 3, 5, 1152, 0, True, False),
    (9, 1100, 6, 1, 5, 1106, 0, True, False), (7, 512, 256, 9, 16, 768, 0, False, False), (5, 40, 8, 300, 16, 48, 0, True, False)])
@pytest.mark.parametrize("pairs", [True, False])
def test_append_shapes(t, dv, dr, heads, block, stride, unaligned, norm, inplace, pairs):
    run_append(t, dv, dr, heads, BF16, BF16, block, stride, pairs, norm, unaligned, seed=t, inplace=inplace)


def test_append_bad_data_and_special_values():
    t, dv, dr = 6, 512, 64
    g = gen(5)
    c, kp = normal(g, t, dv, dtype=BF16), normal(g, t, dr, dtype=BF16)
    c[0, 3], kp[1, 5] = math.nan, math.inf
    cache = torch.zeros(2, 16, dv + dr, device=DEV).to(FP8)
    cs = torch.ones(10, dr, device=DEV)
    slots = torch.tensor([0, 1, 40, 2, 3, -1], device=DEV)
    positions = i32([0, 1, 2, 10, -1, -1])
    err = i32([0])
    sc = torch.tensor([1e-4], device=DEV)  # everything saturates
    binding.append(c, kp, cache, slots, positions, cs, scale=sc, error_flag=err)
    torch.cuda.synchronize()
    assert int(err) == binding.FLAG_PHYS_BLOCK | binding.FLAG_POSITION
    x = cache.float()
    assert x[0, 2:].abs().sum() == 0 and x[1].abs().sum() == 0
    assert math.isnan(x[0, 0, 3]) and x[0, 0].nan_to_num().abs().max() == 448
    pe = x[0, 1, dv:]  # inf turned: inf - b, b + inf saturate, or NaN where both are infinite
    assert (pe.abs() <= 448).logical_or(pe.isnan()).all()
    binding.append(c[:1], kp[:1], cache, slots[:1], positions[:1], cs, norm_weight=torch.ones(dv, device=DEV), scale=sc)
    assert cache.float()[0, 0, :dv].isnan().all()  # a NaN in the row makes its norm NaN


# --- latent_decode -----------------------------------------------------------------

def decode_case(lens, heads, q_len, src, cdt, block, dv=512, dr=64, stride=None, seed=3, scale=0.05, nan_tail=True,
                q_gain=1.0):
    rng = np.random.default_rng(seed)
    g = gen(seed)
    table, blocks = ref.tables(rng, lens, block)
    E = dv + dr
    full = normal(g, blocks, block, stride or E)
    full = ((full / scale).clamp(-448, 448) if cdt == FP8 else full).to(cdt)
    cache = full[:, :, :E]
    if nan_tail:  # slots past a request's end hold anything
        for r, n in enumerate(lens):
            if n > 0 and n % block:
                full[int(table[r, n // block]), n % block:] = math.nan
    q = (normal(g, len(lens), q_len, heads, E) * q_gain).to(src)
    return q, cache, i32(table), i32(lens), (torch.tensor([scale], device=DEV) if cdt == FP8 else None)


def run_decode(case, ws, dv=512, options=0, sm=None, weights_u=None, flag=0):
    q, cache, table, lens, sc = case
    sm = 1.0 / math.sqrt(192) if sm is None else sm
    out = torch.full(q.shape[:3] + (dv,), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    err = i32([0])
    binding.latent_decode(q, cache, table, lens, out, lse, sm_scale=sm, scale=sc, workspace=ws, error_flag=err,
                          options=options)
    torch.cuda.synchronize()
    assert int(err) == flag
    check_decode(case, out, lse, dv, options, sm, weights_u)
    return out, lse


def check_decode(case, out, lse, dv=512, options=0, sm=1.0 / math.sqrt(192), weights_u=None):
    q, cache, table, lens, sc = case
    f = 1.0 if sc is None else float(sc)
    want, wl, pv, worst, flat = ref.decode(q, cache, table, lens, dv, sm, f)
    u, extra, below = ref.U[q.dtype] if weights_u is None else weights_u, 0.0, 0.0
    if cache.dtype == FP8 and options == 0:
        # weights of two e4m3 parts: 2^-8 of their value, and half a subnormal step (2^-10) at 2^6; queries of parts
        # that hold all their bits but those below 2 * 2^-10 where the largest is at least 224
        u, below = 2.0 ** -8, 2.0 ** -16 * flat
        size = cache.double().nan_to_num(0).abs().sum(2).max() * f
        extra = sm * 2.0 ** -16.8 * q.double().abs().amax(3) * size
    ref.check_attention(out, lse, want, wl, pv, worst, q.shape[3], u, extra, below)


GENERAL = binding.OPT_FORCE_GENERAL


@pytest.mark.parametrize("src,cdt", [(BF16, BF16), (F16, F16), (F32, F32), (BF16, FP8), (F16, FP8), (F32, FP8)])
@pytest.mark.parametrize("heads,q_len", [(1, 1), (5, 2), (16, 1)])
def test_decode_general_types(ws, src, cdt, heads, q_len):
    run_decode(decode_case([17, 71, 130, 0, 1], heads, q_len, src, cdt, 16), ws, options=GENERAL, weights_u=0.0)


@pytest.mark.parametrize("dv,dr,block,stride,heads,q_len,lens", [
    (512, 64, 1, 577, 3, 1, [5, 64, 65]), (40, 8, 7, 48, 9, 3, [2, 100, 0, 300]), (1000, 24, 64, 1024, 2, 1, [70]),
    (1, 0, 3, 1, 1, 1, [10, 1]), (128, 0, 64, 128, 130, 2, [129, 64]), (512, 64, 64, 576, 2, 1, [5000, 33])])
def test_decode_general_shapes(ws, dv, dr, block, stride, heads, q_len, lens):
    run_decode(decode_case(lens, heads, q_len, BF16, BF16, block, dv, dr, stride), ws, dv, weights_u=0.0,
               options=GENERAL, sm=1 / math.sqrt(dv + dr))


LENS = [[1], [2, 1, 0], [63, 64, 65], [127, 128, 129, 0, 1], [1000], [17, 71, 130, 0, 3000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads,q_len,src,cdt", [(16, 1, BF16, BF16), (128, 1, BF16, BF16), (64, 2, BF16, FP8),
                                                 (5, 4, F16, F16), (20, 1, F16, FP8), (1, 1, BF16, FP8)])
def test_decode(ws, lens, heads, q_len, src, cdt):
    run_decode(decode_case(lens, heads, q_len, src, cdt, 64), ws)


@pytest.mark.parametrize("block", [8, 16, 24, 32, 48, 128, 200])
@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_decode_page_sizes(ws, block, cdt):
    run_decode(decode_case([700, 3, 65, block, block + 1], 16, 2, BF16, cdt, block, stride=640), ws)


@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_decode_long_and_many(ws, cdt):
    run_decode(decode_case([20011], 16, 1, BF16, cdt, 64), ws)
    rng = np.random.default_rng(11)
    run_decode(decode_case(rng.integers(0, 400, 333).tolist(), 32, 1, BF16, cdt, 32), ws)
    run_decode(decode_case([9000, 1, 300, 12000], 128, 2, BF16, cdt, 64), ws)


@pytest.mark.parametrize("heads,q_len", [(3, 1), (33, 1), (65, 1), (100, 3), (16, 8), (1, 200)])
def test_decode_row_groups(ws, heads, q_len):
    run_decode(decode_case([300, 65, 5], heads, q_len, BF16, BF16, 64), ws)


@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_decode_sharp_scores(ws, cdt):
    """Large scores: the running maximum moves far, and most weights vanish."""
    run_decode(decode_case([2500, 400], 16, 1, BF16, cdt, 64, q_gain=12.0), ws)


@pytest.mark.parametrize("cdt", [BF16, FP8])
def test_decode_growing_scores(ws, cdt):
    """Each tile's scores lie above the last one's, so the running maximum moves at every tile."""
    q, cache, table, lens, sc = decode_case([1500], 16, 1, BF16, cdt, 64, nan_tail=False)
    q[:] = 0.25
    grow = torch.zeros_like(cache, dtype=torch.float32)
    for i in range(24):
        grow[int(table[0, i])] = (i + 1) * 0.125
    cache = grow.to(cdt)
    run_decode((q, cache, table, lens, None), ws, sm=0.2)


def test_decode_bad_pages(ws):
    q, cache, table, lens, sc = decode_case([200, 300, 64], 16, 1, BF16, BF16, 64, nan_tail=False)
    table[0, 1], table[2, 0] = -3, cache.shape[0]
    for options in (0, GENERAL):
        out, lse = run_decode((q, cache, table, lens, sc), ws, flag=binding.FLAG_PHYS_BLOCK, options=options)
        assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    lens[1] = 1000  # past the table's row
    lens[0] = -4
    for options in (0, GENERAL):
        run_decode((q, cache, table, lens, sc), ws, options=options,
                   flag=binding.FLAG_PHYS_BLOCK | binding.FLAG_LOGICAL_BLOCK | binding.FLAG_LENGTH)


def test_decode_strides_stream_graph_and_repeat(ws):
    """Strided q and out, another stream, a captured graph; the same bits every time."""
    q0, cache, table, lens, sc = decode_case([900, 17, 4000], 16, 2, BF16, BF16, 64)
    q = torch.zeros(3, 2, 20, 600, dtype=BF16, device=DEV)[:, :, 2:18, 8:584]
    q.copy_(q0)
    out = torch.zeros(3, 16, 2, 520, dtype=BF16, device=DEV)[:, :, :, 3:515].transpose(1, 2)
    want, _ = run_decode((q, cache, table, lens, sc), ws)
    side, ws2 = torch.cuda.Stream(), torch.empty_like(ws).fill_(255)
    torch.cuda.synchronize()
    binding.latent_decode(q, cache, table, lens, out, None, sm_scale=1 / math.sqrt(192), workspace=ws2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.latent_decode(q, cache, table, lens, out, None, sm_scale=1 / math.sqrt(192), workspace=ws2)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# --- latent_prefill ----------------------------------------------------------------

def prefill_case(q_lens, k_lens, heads, dtype, dn=128, dr=64, dv=128, prev=False, seed=3, pad=0, gain=1.0):
    g = gen(seed)
    tq, tk = sum(q_lens), sum(k_lens)
    q = (normal(g, tq, heads, dn + dr + pad) * gain).to(dtype)[:, :, :dn + dr]
    kv = normal(g, tk, heads, dn + dv + pad, dtype=dtype)
    pe = normal(g, tk, 512 + dr + pad, dtype=dtype)[:, 512:512 + dr]
    c = dict(q=q, k=kv[:, :, :dn], v=kv[:, :, dn:dn + dv], pe=pe, cu_q=i32(np.cumsum([0] + list(q_lens))),
             cu_k=i32(np.cumsum([0] + list(k_lens))))
    if prev:
        c["prev_out"], c["prev_lse"] = normal(g, tq, heads, dv, dtype=dtype), 4 + normal(g, tq, heads)
        c["prev_lse"][::3] = -math.inf
        c["prev_out"][::3] = math.nan  # a state that holds nothing yet
    return c


def run_prefill(c, ws, causal, options=0, weights_u=None, sm=None, inplace=False):
    q, v = c["q"], c["v"]
    sm = 1 / math.sqrt(q.shape[2]) if sm is None else sm
    want, wl, pv, worst = ref.prefill(q, c["k"], c["pe"], v, c["cu_q"], c["cu_k"], sm, causal, c.get("prev_out"),
                                      c.get("prev_lse"))
    out = torch.full((q.shape[0], q.shape[1], v.shape[2]), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    if inplace:
        out, lse = c["prev_out"], c["prev_lse"]
    err = i32([0])
    binding.latent_prefill(q, c["k"], c["pe"], v, c["cu_q"], c["cu_k"], out, lse, sm_scale=sm, causal=causal,
                           prev_out=c.get("prev_out"), prev_lse=c.get("prev_lse"), workspace=ws, error_flag=err,
                           options=options)
    torch.cuda.synchronize()
    assert int(err) == 0
    u = ref.U[q.dtype] if weights_u is None else weights_u
    ref.check_attention(out, lse, want, wl, pv, worst, q.shape[2], u)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("prev", [False, True])
def test_prefill_general(ws, dtype, causal, prev):
    run_prefill(prefill_case([17, 0, 40, 1], [17, 5, 70, 33], 3, dtype, prev=prev), ws, causal, GENERAL, 0.0)


@pytest.mark.parametrize("dn,dr,dv,pad", [(40, 8, 24, 1), (1, 0, 1, 0), (512, 64, 512, 0), (128, 64, 128, 3), (64, 64, 1000, 0)])
def test_prefill_general_shapes(ws, dn, dr, dv, pad):
    run_prefill(prefill_case([9, 33], [50, 33], 2, BF16, dn, dr, dv, pad=pad), ws, True, GENERAL, weights_u=0.0)


Q_K = [([1], [1]), ([17, 71, 130, 0], [17, 71, 130, 0]), ([128], [128]), ([256, 1], [300, 500]), ([257], [129]),
       ([1, 2, 3], [0, 2, 129]), ([100], [3001]), ([700, 5], [900, 5])]


@pytest.mark.parametrize("q_lens,k_lens", Q_K)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,heads", [(BF16, 2), (F16, 3)])
def test_prefill(ws, q_lens, k_lens, causal, dtype, heads):
    run_prefill(prefill_case(q_lens, k_lens, heads, dtype), ws, causal)


@pytest.mark.parametrize("causal", [False, True])
def test_prefill_joined(ws, causal):
    c = prefill_case([300, 0, 77], [1000, 3, 500], 4, BF16, prev=True)
    a = run_prefill(c, ws, causal)
    b = run_prefill(c, ws, causal, inplace=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("causal", [False, True])
def test_prefill_split(ws, causal):
    """Few rows over many keys, and more pieces than SMs: shares cut requests."""
    run_prefill(prefill_case([64], [20000], 2, BF16, prev=True), ws, causal)
    run_prefill(prefill_case([1500, 900], [1500, 2100], 5, BF16), ws, causal)


def test_prefill_sharp_scores(ws):
    run_prefill(prefill_case([300], [900], 2, BF16, gain=12.0), ws, False)


def test_prefill_chunks_equal_the_whole(ws):
    """A context taken in two calls joined by the state equals one call, within both calls' roundings."""
    c = prefill_case([200], [1200], 2, BF16)
    whole, lse = run_prefill(c, ws, True)
    first = dict(c, k=c["k"][:1000], v=c["v"][:1000], pe=c["pe"][:1000], cu_k=i32([0, 1000]))
    out1, lse1 = run_prefill(first, ws, False)
    rest = dict(c, k=c["k"][1000:], v=c["v"][1000:], pe=c["pe"][1000:], cu_k=i32([0, 200]), prev_out=out1,
                prev_lse=lse1)
    out2, lse2 = run_prefill(rest, ws, True)
    assert (lse2 - lse).abs().max() < 1e-3
    assert (out2.float() - whole.float()).abs().max() <= 6 * 2.0 ** -8 * c["v"].float().abs().max()


def test_prefill_order_errors(ws):
    c = prefill_case([10, 10], [10, 10], 1, BF16)
    c["cu_q"] = i32([0, 12, 10])
    out = torch.full((20, 1, 128), 7.0, dtype=BF16, device=DEV)
    for options in (0, GENERAL):
        err = i32([0])
        binding.latent_prefill(c["q"], c["k"], c["pe"], c["v"], c["cu_q"], c["cu_k"], out, None, sm_scale=0.1,
                               workspace=ws, error_flag=err, options=options)
        assert int(err) == binding.FLAG_CU_ORDER and (out[12:] == 7).all() and not (out[:12] == 7).any()


def test_prefill_nan_past_a_request(ws):
    """Keys of other requests and rows past the last key do not reach a request's result."""
    c = prefill_case([70, 70], [100, 100], 2, BF16)
    kv = torch.full((300, 2, 256), math.nan, dtype=BF16, device=DEV)
    kv[:200, :, :128], kv[:200, :, 128:] = c["k"], c["v"]
    kv[100:200] = math.nan
    pe = torch.full((300, 64), math.nan, dtype=BF16, device=DEV)
    pe[:100] = c["pe"][:100]
    for options in (0, GENERAL):
        out = torch.zeros(140, 2, 128, dtype=BF16, device=DEV)
        binding.latent_prefill(c["q"], kv[:, :, :128], pe, kv[:, :, 128:], c["cu_q"], c["cu_k"], out, None,
                               sm_scale=0.1, workspace=ws, options=options)
        assert not out[:70].isnan().any()

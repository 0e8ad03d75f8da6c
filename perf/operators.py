"""Measured cases of the latent-attention operators.

Four operators around the paged cache, each in two forms: the framework's
calls (`own` true) and plain torch operations in 32 bits (`own` false).

  plan     block tables, slots and positions of one serving step from the
           request lengths (binding.plan_step)
  append   latent norm, rotation of the shared key part and of the queries,
           and the write into the paged cache (binding.append)
  decode   absorbed latent attention of one or a few new tokens a request over
           the paged cache (binding.latent_decode)
  prefill  expanded latent attention of a chunk of new tokens, joined with the
           state of earlier keys (binding.latent_prefill)

A cache entry is 512 latent values and 64 rotated ones (576); expanded heads
have 128 + 64 query and key values and 128 values.
"""
import math
import random

import torch

own = False

LATENT = 512      # latent values of an entry
ROPE = 64         # rotated values of an entry
ENTRY = LATENT + ROPE
NOPE = 128        # unrotated key values of an expanded head
VALUE = 128       # values of an expanded head
POSITIONS = 65536 # rows of the rotation table
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
EPS = 1e-6

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1}


# --- the cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step's bookkeeping: 64 requests, one token each
        {"name": "plan 64 x 1 token", "op": "plan", "reqs": 64, "ctx_lo": 1, "ctx_hi": 32768, "new_lo": 1, "new_hi": 1,
         "block": 64},
        # a prefill-heavy step of many requests on small pages
        {"name": "plan 2048 ragged", "op": "plan", "reqs": 2048, "ctx_lo": 0, "ctx_hi": 4096, "new_lo": 1,
         "new_hi": 512, "block": 16},
        # the cache write of one decode step
        {"name": "append 64 tokens", "op": "append", "tokens": 64, "heads": 16, "src": "bf16", "cache": "bf16",
         "stride": ENTRY, "pairs": True, "padding": 0, "block": 64},
        # fp16, odd sizes, padded cache rows, halves rotated, padding tokens of a captured graph
        {"name": "append 1237 odd fp16", "op": "append", "tokens": 1237, "heads": 5, "src": "fp16", "cache": "fp16",
         "stride": 640, "pairs": False, "padding": 43, "block": 16},
        # a prefill chunk quantised into an fp8 cache, all heads of a wide model
        {"name": "append 8192 fp8", "op": "append", "tokens": 8192, "heads": 128, "src": "bf16", "cache": "fp8",
         "stride": ENTRY, "pairs": True, "padding": 0, "block": 64},
        # a few short requests, one of them empty: latency
        {"name": "decode short", "op": "decode", "lens": "17,71,130,0", "heads": 16, "q_len": 1, "src": "bf16",
         "cache": "bf16", "stride": ENTRY, "block": 64},
        # one long request: everything hangs on the split over the cache
        {"name": "decode one 60000", "op": "decode", "lens": "60000", "heads": 16, "q_len": 1, "src": "bf16",
         "cache": "bf16", "stride": ENTRY, "block": 64},
        # skewed requests, fp8 cache, two tokens each (one drafted)
        {"name": "decode skew 8 fp8", "op": "decode", "lens": "32768,17,71,4096,1,513,0,8191", "heads": 64, "q_len": 2,
         "src": "bf16", "cache": "fp8", "stride": ENTRY, "block": 64},
        # a full decode batch of a wide model, padded rows
        {"name": "decode ragged 64 x 128 heads", "op": "decode", "reqs": 64, "lo": 1, "hi": 32768, "heads": 128,
         "q_len": 1, "src": "bf16", "cache": "bf16", "stride": 640, "block": 64},
        # short prompts, one empty
        {"name": "prefill short", "op": "prefill", "q_lens": "17,71,130,0", "k_lens": "17,71,130,0", "heads": 16,
         "src": "bf16", "causal": True, "prev": False},
        # a chunk of new tokens over a gathered context, joined with its own causal part
        {"name": "prefill 512 over 60000", "op": "prefill", "q_lens": "512", "k_lens": "60000", "heads": 16,
         "src": "bf16", "causal": False, "prev": True},
        # one long prompt
        {"name": "prefill causal 8192", "op": "prefill", "q_lens": "8192", "k_lens": "8192", "heads": 32,
         "src": "bf16", "causal": True, "prev": False},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "prefill", "prefill"])
    if op == "plan":
        hi = rng.choice([1, 4, _log(rng, 1, 512)])
        return {"op": op, "reqs": _log(rng, 1, 4096), "ctx_lo": 0, "ctx_hi": _log(rng, 1, 8192), "new_lo": rng.choice([0, 1]),
                "new_hi": hi, "block": rng.choice([16, 32, 64, 128])}
    if op == "append":
        src = rng.choice(["bf16", "bf16", "fp16"])
        tokens = _log(rng, 1, 8192)
        return {"op": op, "tokens": tokens, "heads": _log(rng, 1, 128), "src": src, "cache": rng.choice([src, "fp8"]),
                "stride": rng.choice([ENTRY, 640]), "pairs": rng.random() < 0.5, "padding": rng.choice([0, tokens // 9]),
                "block": rng.choice([16, 32, 64, 128])}
    if op == "decode":
        src = rng.choice(["bf16", "bf16", "fp16"])
        heads, q_len, reqs = rng.choice([1, 5, 8, 16, 20, 32, 64, 128]), rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 64)
        most = min(60000, 100000000 // (heads * q_len * reqs), 2000000 // reqs)
        return {"op": op, "reqs": reqs, "lo": 1, "hi": _log(rng, 16, max(16, most)), "heads": heads, "q_len": q_len,
                "src": src, "cache": rng.choice([src, src, "fp8"]), "stride": rng.choice([ENTRY, 640]),
                "block": rng.choice([16, 32, 64, 128])}
    heads, reqs = rng.choice([1, 3, 8, 16, 32, 128]), _log(rng, 1, 8)
    most = 1000000000 // (heads * reqs)
    keys = min(60000, 960000 // (heads * reqs))
    q = _log(rng, 1, min(8192, keys, int(math.sqrt(most))))
    causal = rng.random() < 0.5
    k = _log(rng, q, max(q, min(keys, most // q)))
    lens = [(_log(rng, 1, q), _log(rng, 1, k)) for _ in range(reqs - 1)] + [(q, k)]
    lens = [(a, max(a, b)) for a, b in lens]
    return {"op": op, "q_lens": ",".join(str(a) for a, _ in lens), "k_lens": ",".join(str(b) for _, b in lens),
            "heads": heads, "src": rng.choice(["bf16", "bf16", "fp16"]), "causal": causal, "prev": rng.random() < 0.4}


def _lens(case):
    """The request lengths of a decode case: listed, or spread by the case's own values."""
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    rng = random.Random("%d %d %d" % (case["reqs"], case["lo"], case["hi"]))
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["reqs"])]


def _plan_lens(case):
    rng = random.Random("%d %d %d %d" % (case["reqs"], case["ctx_hi"], case["new_hi"], case["block"]))
    ctx = [_log(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["reqs"])]
    return ctx, new


def _prefill_lens(case):
    return [int(x) for x in case["q_lens"].split(",")], [int(x) for x in case["k_lens"].split(",")]


def _pages(length, block):
    return -(-length // block)


def _seen(q, k, causal):
    """Pairs of a query and a key that it sees: query i of q sees the first k - q + i + 1 keys."""
    if not causal:
        return q * k
    first = k - q + 1
    lo = max(0, -first + 1) if first <= 0 else 0  # queries that see nothing
    n = q - lo
    return n * (first + lo + k) // 2 if n > 0 else 0


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _plan_lens(case)
        t, r, b = sum(new), case["reqs"], case["block"]
        taken = sum(_pages(c + n, b) - _pages(c, b) for c, n in zip(ctx, new))
        # lengths in; prefix sums and lengths out; ids taken and written; slot, position and request of each token;
        # the last page of each request
        return {"bytes": 4 * (2 * r + 3 * r + 2 + 2 * taken + r) + 16 * t, "flops": 0}
    if op == "append":
        t, real, s, d = case["tokens"], case["tokens"] - case["padding"], BYTES[case["src"]], BYTES[case["cache"]]
        return {"bytes": real * (ENTRY * (s + d) + 2 * case["heads"] * ROPE * s + 4 * ROPE) + 12 * t + 4 * LATENT,
                "flops": real * (4 * LATENT + 6 * ROPE * (1 + case["heads"]))}
    if op == "decode":
        lens, rows = _lens(case), case["heads"] * case["q_len"]
        n, s = sum(lens), BYTES[case["src"]]
        pages = sum(_pages(x, case["block"]) for x in lens)
        return {"bytes": n * ENTRY * BYTES[case["cache"]] + len(lens) * rows * ((ENTRY + LATENT) * s + 4) + 4 * pages,
                "flops": 2 * rows * n * (ENTRY + LATENT)}
    qs, ks = _prefill_lens(case)
    h, s = case["heads"], BYTES[case["src"]]
    qb = h * (NOPE + ROPE + VALUE) * s + 4 * h + (h * (VALUE * s + 4) if case["prev"] else 0)
    return {"bytes": sum(qs) * qb + sum(ks) * (h * (NOPE + VALUE) + ROPE) * s,
            "flops": 2 * h * sum(_seen(a, b, case["causal"]) for a, b in zip(qs, ks)) * (NOPE + ROPE + VALUE)}


# --- the inputs ------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _sums(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), _i32(lens).cumsum(0, dtype=torch.int32)])


def _entries(g, blocks, block, stride, dtype, scale):
    """A cache of N(0, 1) entries; an fp8 one holds them divided by its scale."""
    values = torch.empty((blocks, block, stride), dtype=TYPES[dtype], device="cuda")
    step = max(1, (1 << 26) // (block * stride))
    for i in range(0, blocks, step):
        x = _normal(g, min(step, blocks - i), block, stride)
        values[i:i + step] = ((x / scale).clamp(-448, 448) if dtype == "fp8" else x).to(TYPES[dtype])
    return values[:, :, :ENTRY]


def _table(g, lens, block, width, spare=64):
    """Block ids of shuffled pages; unused columns are -1. Returns the table and the `spare` ids left."""
    need = torch.tensor([_pages(x, block) for x in lens], device="cuda")
    total = int(need.sum())
    ids = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    column = torch.arange(width, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + column
    table = torch.where(column < need[:, None], ids[at.clamp(max=total + spare - 1)], -1)
    return table.to(torch.int32).contiguous(), ids[total:]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"op": op, "seen": case}
    if op == "plan":
        ctx, new = _plan_lens(case)
        b, r, t = case["block"], case["reqs"], max(1, sum(new))
        width = max(1, max(_pages(c + n, b) for c, n in zip(ctx, new)))
        taken = sum(_pages(c + n, b) - _pages(c, b) for c, n in zip(ctx, new))
        table, free = _table(g, ctx, b, width, taken + 7)
        s["num_blocks"] = sum(_pages(c, b) for c in ctx) + taken + 7
        s.update(table=table, free=free.contiguous(), ctx=_i32(ctx), new=_i32(new), block=b)
        s.update(slots=torch.empty(t, dtype=torch.int64, device="cuda"), positions=torch.empty(t, dtype=torch.int32, device="cuda"),
                 token_to_seq=torch.empty(t, dtype=torch.int32, device="cuda"), cu_new=torch.empty(r + 1, dtype=torch.int32, device="cuda"),
                 seq_lens=torch.empty(r, dtype=torch.int32, device="cuda"), cu_seq=torch.empty(r + 1, dtype=torch.int32, device="cuda"),
                 taken=torch.empty(1, dtype=torch.int32, device="cuda"))
        return s
    if op == "append":
        t, h, src, b = case["tokens"], case["heads"], TYPES[case["src"]], case["block"]
        blocks = _pages(t, b) + 5
        # the down-projection's output: latent and shared key part side by side; queries of the up-projection
        down = _normal(g, t, ENTRY, dtype=src)
        s.update(c_kv=down[:, :LATENT], k_pe=down[:, LATENT:], weight=1 + 0.1 * _normal(g, LATENT))
        s["q_pe"] = _normal(g, t, h, NOPE + ROPE, dtype=src)[:, :, NOPE:]
        s["q_full"] = torch.zeros((t, h, ENTRY), dtype=src, device="cuda")
        s["q_out"] = s["q_full"][:, :, LATENT:]
        s["cache"] = torch.zeros((blocks, b, case["stride"]), dtype=TYPES[case["cache"]], device="cuda")[:, :, :ENTRY]
        s["scale"] = torch.tensor([0.05], device="cuda") if case["cache"] == "fp8" else None
        s["slots"] = torch.randperm(blocks * b, generator=g, device="cuda")[:t]
        s["positions"] = torch.randint(0, POSITIONS, (t,), generator=g, device="cuda", dtype=torch.int32)
        if case["padding"]:
            s["slots"][-case["padding"]:] = -1
            s["positions"][-case["padding"]:] = -1
        angle = torch.arange(POSITIONS, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(ROPE // 2, dtype=torch.float64, device="cuda") / (ROPE // 2))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["pairs"] = case["pairs"]
        return s
    if op == "decode":
        lens, b, src = _lens(case), case["block"], TYPES[case["src"]]
        width = max(1, max(_pages(x, b) for x in lens))
        blocks = sum(_pages(x, b) for x in lens) + 64
        s["table"], _ = _table(g, lens, b, width)
        s["scale"] = torch.tensor([0.05], device="cuda") if case["cache"] == "fp8" else None
        s["cache"] = _entries(g, blocks, b, case["stride"], case["cache"], 0.05)
        s["q"] = _normal(g, len(lens), case["q_len"], case["heads"], ENTRY, dtype=src)
        s["seq_lens"] = _i32(lens)
        s["out"] = torch.empty((len(lens), case["q_len"], case["heads"], LATENT), dtype=src, device="cuda")
        s["lse"] = torch.empty((len(lens), case["q_len"], case["heads"]), device="cuda")
        return s
    qs, ks = _prefill_lens(case)
    h, src, tq, tk = case["heads"], TYPES[case["src"]], sum(qs), sum(ks)
    s["q"] = _normal(g, tq, h, NOPE + ROPE, dtype=src)
    # the up-projection's output: keys and values side by side; the shared key part as the gather leaves it
    kv = _normal(g, tk, h, NOPE + VALUE, dtype=src)
    s["k"], s["v"] = kv[:, :, :NOPE], kv[:, :, NOPE:]
    s["k_pe"] = _normal(g, tk, ENTRY, dtype=src)[:, LATENT:]
    s["cu_q"], s["cu_k"] = _sums(qs), _sums(ks)
    s["max_q"], s["max_k"], s["causal"] = max(qs), max(ks), case["causal"]
    if case["prev"]:
        s["prev_out"] = _normal(g, tq, h, VALUE, dtype=src) * 0.1
        s["prev_lse"] = 5 + _normal(g, tq, h)
    s["out"] = torch.empty((tq, h, VALUE), dtype=src, device="cuda")
    s["lse"] = torch.empty((tq, h), device="cuda")
    return s


# --- one pass --------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _own_plan(s):
    from paged_mla_kv_cache_gb300 import binding
    binding.plan_step(s["ctx"], s["new"], s["table"], s["free"], s["block"], s["slots"], s["positions"],
                      s["token_to_seq"], s["cu_new"], s["seq_lens"], s["cu_seq"], s["taken"], s["num_blocks"])
    return [s["table"], s["slots"], s["positions"], s["token_to_seq"], s["cu_new"], s["seq_lens"], s["cu_seq"], s["taken"]]


def _own_append(s):
    from paged_mla_kv_cache_gb300 import binding
    binding.append(s["c_kv"], s["k_pe"], s["cache"], s["slots"], s["positions"], s["cos_sin"], norm_weight=s["weight"],
                   eps=EPS, scale=s["scale"], q_pe=s["q_pe"], q_out=s["q_out"], interleaved=s["pairs"])
    return [s["cache"], s["q_out"]]


def _own_decode(s):
    from paged_mla_kv_cache_gb300 import binding
    if "workspace" not in s:  # kept by a serving loop
        s["workspace"] = binding.new_attention_workspace("cuda")
    binding.latent_decode(s["q"], s["cache"], s["table"], s["seq_lens"], s["out"], s["lse"], sm_scale=SCALE,
                          scale=s["scale"], workspace=s["workspace"])
    return [s["out"], s["lse"]]


def _own_prefill(s):
    from paged_mla_kv_cache_gb300 import binding
    if "workspace" not in s:
        s["workspace"] = binding.new_attention_workspace("cuda")
    binding.latent_prefill(s["q"], s["k"], s["k_pe"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["lse"], sm_scale=SCALE,
                           causal=s["causal"], prev_out=s.get("prev_out"), prev_lse=s.get("prev_lse"),
                           workspace=s["workspace"])
    return [s["out"], s["lse"]]


def _plain_plan(s):
    ctx, new, b = s["ctx"].long(), s["new"].long(), s["block"]
    end = ctx + new
    zero = ctx.new_zeros(1)
    cu = torch.cat([zero, new.cumsum(0)])
    first = (ctx + b - 1) // b
    need = (end + b - 1) // b - first
    before = need.cumsum(0) - need
    column = torch.arange(s["table"].shape[1], device=ctx.device)
    fresh = (column >= first[:, None]) & (column < (first + need)[:, None])
    table = torch.where(fresh, s["free"][(before[:, None] + column - first[:, None]).clamp(0, s["free"].shape[0] - 1)], s["table"])
    t = torch.arange(s["slots"].shape[0], device=ctx.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    real = seq < ctx.shape[0]
    seq = seq.clamp(max=ctx.shape[0] - 1)
    position = ctx[seq] + t - cu[seq]
    slots = table[seq, (position // b).clamp(max=table.shape[1] - 1)].long() * b + position % b
    return [table, torch.where(real, slots, -1), torch.where(real, position, -1).int(), torch.where(real, seq, -1).int(),
            cu.int(), end.int(), torch.cat([zero, end.cumsum(0)]).int(), need.sum().int().view(1)]


def _rotate(x, cos, sin, pairs):
    """x [..., ROPE] in 32 bits: pairs (2i, 2i + 1), or (i, i + ROPE / 2)."""
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    p, q = a * cos - b * sin, b * cos + a * sin
    return torch.stack([p, q], -1).flatten(-2) if pairs else torch.cat([p, q], -1)


def _plain_append(s):
    cache, b = s["cache"], s["cache"].shape[1]
    c = s["c_kv"].float()
    latent = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"]
    cs = s["cos_sin"][s["positions"].long().clamp(min=0)]
    cos, sin = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    entry = torch.cat([latent, _rotate(s["k_pe"].float(), cos, sin, s["pairs"])], 1)
    if s["scale"] is not None:
        entry = (entry / s["scale"]).clamp(-448, 448)
    real = s["slots"] >= 0
    slot, entry = s["slots"][real], entry[real]
    cache[slot // b, slot % b] = entry.to(cache.dtype)
    q = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None], s["pairs"]).to(s["q_out"].dtype)
    seen = s["positions"] >= 0
    s["q_out"][seen] = q[seen]
    return [cache, s["q_out"]]


def _attend(scores, seen, values):
    """Softmax over the last axis where `seen`; rows that see nothing give 0 and a log-sum of -inf."""
    scores = torch.where(seen, scores, -math.inf)
    most = scores.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    p = torch.exp(scores - most)
    total = p.sum(-1, keepdim=True)
    out = values(p) / torch.where(total == 0, 1.0, total)
    return out, (most + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    q, cache, table = s["q"].float(), s["cache"], s["table"]
    n, q_len, h, _ = q.shape
    kv = cache[table.clamp(min=0).long()].reshape(n, -1, ENTRY).float()
    if s["scale"] is not None:
        kv = kv * s["scale"]
    place = torch.arange(kv.shape[1], device=q.device)
    last = s["seq_lens"][:, None] - q_len + 1 + torch.arange(q_len, device=q.device)  # keys that a query sees
    seen = (place < last[:, :, None])[:, :, None].expand(n, q_len, h, -1).reshape(n, q_len * h, -1)
    scores = torch.bmm(q.view(n, q_len * h, ENTRY), kv.transpose(1, 2)) * SCALE
    out, lse = _attend(scores, seen, lambda p: torch.bmm(p, kv[:, :, :LATENT]))
    return [out.view(n, q_len, h, LATENT).to(s["out"].dtype), lse.view(n, q_len, h)]


def _plain_prefill(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q.diff(), cu_k.diff()
    iq, ik = torch.arange(s["max_q"], device=lq.device), torch.arange(s["max_k"], device=lq.device)
    at_q = (cu_q[:-1, None] + iq).clamp(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp(max=s["v"].shape[0] - 1)
    q = s["q"][at_q].float().transpose(1, 2)                                                   # [n, h, q, 192]
    k = s["k"][at_k].float().transpose(1, 2)                                                   # [n, h, k, 128]
    v = s["v"][at_k].float().transpose(1, 2)
    pe = s["k_pe"][at_k].float()[:, None]                                                      # shared by the heads
    scores = q[..., :NOPE] @ k.transpose(-1, -2)
    scores += q[..., NOPE:] @ pe.transpose(-1, -2)
    scores *= SCALE
    seen = ik < lk[:, None, None]
    if s["causal"]:
        seen = seen & (ik <= (iq + (lk - lq)[:, None])[:, :, None])
    out, lse = _attend(scores, seen[:, None], lambda p: p @ v)
    real = iq < lq[:, None]
    out, lse = out.transpose(1, 2)[real], lse.transpose(1, 2)[real]                            # rows in the order of q
    if "prev_lse" in s:
        both = torch.logaddexp(lse, s["prev_lse"])
        out = out * torch.exp(lse - both)[..., None] + s["prev_out"].float() * torch.exp(s["prev_lse"] - both)[..., None]
        lse = both
    return [out.to(s["out"].dtype), lse]


_run_own = {"plan": _own_plan, "append": _own_append, "decode": _own_decode, "prefill": _own_prefill}
_run_plain = {"plan": _plain_plan, "append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}


# --- the definition in 64 bits ------------------------------------------------------

def _exact_rotation(x, positions, pairs):
    half = ROPE // 2
    angle = positions.double()[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    turn = torch.polar(torch.ones_like(angle), angle).view((len(x),) + (1,) * (x.dim() - 2) + (half,))
    x = x.double()
    z = torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) if pairs else torch.complex(x[..., :half], x[..., half:])
    z = z * turn
    return torch.view_as_real(z).flatten(-2) if pairs else torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "append":
        real = torch.nonzero(s["slots"] >= 0).flatten()
        c = s["c_kv"][real].double()
        latent = c / (c.square().mean(1, keepdim=True) + EPS).sqrt() * s["weight"].double()
        entry = torch.cat([latent, _exact_rotation(s["k_pe"][real], s["positions"][real], s["pairs"])], 1)
        if s["scale"] is not None:
            entry = torch.clamp(entry / s["scale"].double(), -448, 448)
        cache = torch.zeros(s["cache"].shape, dtype=torch.float64, device="cuda")
        cache.view(-1, ENTRY)[s["slots"][real]] = entry
        q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
        q[real] = _exact_rotation(s["q_pe"][real], s["positions"][real], s["pairs"])
        return [cache, q]
    if op == "decode":
        outs, lses = [], []
        factor = 1.0 if s["scale"] is None else s["scale"].double()
        for r, n in enumerate(_lens(case)):
            q = s["q"][r].double()
            pages = s["table"][r, :_pages(n, case["block"])].long()
            kv = s["cache"][pages].reshape(-1, ENTRY)[:n].double() * factor
            out = torch.zeros(q.shape[:2] + (LATENT,), dtype=torch.float64, device="cuda")
            lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
            for i in range(q.shape[0]):
                m = n - q.shape[0] + 1 + i
                if m > 0:
                    x = q[i] @ kv[:m].T * SCALE
                    lse[i] = torch.logsumexp(x, 1)
                    out[i] = torch.exp(x - lse[i][:, None]) @ kv[:m, :LATENT]
            outs.append(out)
            lses.append(lse)
        return [torch.stack(outs), torch.stack(lses)]
    qs, ks = _prefill_lens(case)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    a = b = 0
    for nq, nk in zip(qs, ks):
        for h in range(case["heads"]):
            if nq == 0 or nk == 0:
                continue
            key = torch.cat([s["k"][b:b + nk, h], s["k_pe"][b:b + nk]], 1).double()
            x = s["q"][a:a + nq, h].double() @ key.T * SCALE
            if case["causal"]:
                x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(nk - nq + 1), -math.inf)
            z = torch.logsumexp(x, 1)
            lse[a:a + nq, h] = z
            out[a:a + nq, h] = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None]) @ s["v"][b:b + nk, h].double()
        a, b = a + nq, b + nk
    if case["prev"]:
        w = torch.sigmoid(lse - s["prev_lse"].double())[..., None]  # the share of these keys
        out = w * out + (1 - w) * s["prev_out"].double()
        lse = torch.maximum(lse, s["prev_lse"].double()) + torch.log1p(torch.exp(-(lse - s["prev_lse"].double()).abs()))
    return [out, lse]

"""Measured cases of sparse and shared-prefix attention over the paged latent cache.

Two ways to spend less on long contexts, each in two forms: the framework's
calls (`own` true) and plain torch operations in 32 bits (`own` false).

  bounds   largest and smallest value of each column of a page's entries, kept
           up to date as entries join (binding.block_bounds)
  scores   an upper bound of every page's scores for each new token, from those
           (binding.block_scores)
  sparse   the best pages of each token (binding.select_blocks) and absorbed
           attention over them (binding.latent_decode)
  shared   absorbed attention of requests that share a long prefix, which is
           read once for all of them (binding.latent_decode_shared)

A cache entry is 512 latent values and 64 rotated ones (576).
"""
import math
import random

import torch

own = False

LATENT = 512      # latent values of an entry
ROPE = 64         # rotated values of an entry
ENTRY = LATENT + ROPE
SCALE = 1.0 / math.sqrt(128 + 64)
FP8_SCALE = 0.05

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp8": 1}


# --- the cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 requests: one entry joins a page of each
        {"name": "bounds step of 64", "op": "bounds", "reqs": 64, "ctx_lo": 1, "ctx_hi": 32768, "new_lo": 1, "new_hi": 1,
         "src": "bf16", "cache": "bf16", "stride": ENTRY, "block": 64},
        # chunks of prompts on small pages, padded rows, some pages begun before
        {"name": "bounds 37 ragged fp16", "op": "bounds", "reqs": 37, "ctx_lo": 0, "ctx_hi": 4096, "new_lo": 1,
         "new_hi": 512, "src": "fp16", "cache": "fp16", "stride": 640, "block": 16},
        # a long context written at once, e4m3 entries
        {"name": "bounds 300000 fp8", "op": "bounds", "reqs": 1, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 300000,
         "new_hi": 300000, "src": "bf16", "cache": "fp8", "stride": ENTRY, "block": 64},
        # a few short requests, one of them empty: latency
        {"name": "scores short", "op": "scores", "lens": "17,71,130,0", "heads": 16, "q_len": 1, "src": "bf16",
         "cache": "bf16", "block": 64, "lse": False},
        # one long request of an e4m3 cache on small pages, two tokens (one drafted), weights instead of scores
        {"name": "scores 60000 fp8 with lse", "op": "scores", "lens": "60000", "heads": 16, "q_len": 2, "src": "fp16",
         "cache": "fp8", "block": 32, "lse": True},
        # the largest decode batch of a wide model, no request short
        {"name": "scores ragged 256 x 128 heads", "op": "scores", "reqs": 256, "lo": 1024, "hi": 32768, "heads": 128,
         "q_len": 1, "src": "bf16", "cache": "bf16", "block": 64, "lse": True},
        # a few short requests on small pages: latency
        {"name": "sparse short", "op": "sparse", "lens": "17,71,130,0", "heads": 16, "q_len": 1, "src": "bf16",
         "cache": "bf16", "stride": ENTRY, "block": 16, "keep": 4, "first": 1, "last": 1},
        # one long request, two tokens that choose their own pages, e4m3 cache
        {"name": "sparse 60000 fp8", "op": "sparse", "lens": "60000", "heads": 20, "q_len": 2, "src": "bf16",
         "cache": "fp8", "stride": ENTRY, "block": 64, "keep": 37, "first": 1, "last": 3},
        # a full decode batch of a wide model, padded rows
        {"name": "sparse ragged 64 x 128 heads", "op": "sparse", "reqs": 64, "lo": 1, "hi": 32768, "heads": 128,
         "q_len": 1, "src": "bf16", "cache": "bf16", "stride": 640, "block": 64, "keep": 32, "first": 1, "last": 2},
        # a few requests behind a short system prompt
        {"name": "shared short", "op": "shared", "groups": "4", "alone": 0, "prefix": "513", "lo": 1, "hi": 130, "heads": 16,
         "q_len": 1, "src": "bf16", "cache": "bf16", "stride": ENTRY, "block": 64},
        # two prompts, an empty group, a request behind none; e4m3 cache, drafted tokens
        {"name": "shared 16 in groups fp8", "op": "shared", "groups": "5,0,11", "alone": 1, "prefix": "8191,71,32768",
         "lo": 2, "hi": 513, "heads": 20, "q_len": 2, "src": "bf16", "cache": "fp8", "stride": ENTRY, "block": 64},
        # a full decode batch of a wide model behind one long document, padded rows
        {"name": "shared 64 x 128 heads over 32768", "op": "shared", "groups": "64", "alone": 0, "prefix": "32768", "lo": 1,
         "hi": 1024, "heads": 128, "q_len": 1, "src": "bf16", "cache": "bf16", "stride": 640, "block": 64},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)))))))


def draw(rng):
    op = rng.choice(["bounds", "scores", "scores", "sparse", "sparse", "shared", "shared", "shared"])
    src = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([src, src, "fp8"])
    block = rng.choice([16, 32, 64, 128])
    stride = rng.choice([ENTRY, 640])
    if op == "bounds":
        reqs = _log(rng, 1, 256)
        return {"op": op, "reqs": reqs, "ctx_lo": 0, "ctx_hi": _log(rng, 1, 400000 // reqs), "new_lo": rng.choice([0, 1]),
                "new_hi": rng.choice([1, 4, _log(rng, 1, 200000 // reqs)]), "src": src, "cache": cache, "stride": stride,
                "block": block}
    heads = rng.choice([1, 5, 8, 16, 20, 32, 64, 128])
    if op in ("scores", "sparse"):
        q_len, reqs = rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 256 if op == "scores" else 64)
        most = min(60000, 100000000 // (heads * q_len * reqs), 1000000 // reqs)
        case = {"op": op, "reqs": reqs, "lo": 1, "hi": _log(rng, 16, max(16, most)), "heads": heads, "q_len": q_len,
                "src": src, "cache": cache, "block": block}
        if op == "scores":
            return {**case, "lse": rng.random() < 0.5}
        first, last = rng.choice([0, 1, 2]), rng.choice([1, 1, 2, 4])
        return {**case, "stride": stride, "keep": first + last + _log(rng, 1, 64), "first": first, "last": last}
    q_len, groups = rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 8)
    members = [rng.choice([0, 1]) if rng.random() < 0.2 else _log(rng, 1, 64 // groups) for _ in range(groups)]
    widest = max(1, max(members)) * heads * q_len  # rows of the largest group: the plain form pads the others to it
    most = min(60000, 200000000 // (widest * groups), 400000 // groups)
    return {"op": op, "groups": ",".join(map(str, members)), "alone": 0 if max(members) else 1,
            "prefix": ",".join(str(_log(rng, 16, max(16, most))) for _ in members), "lo": q_len,
            "hi": _log(rng, q_len, 1024), "heads": heads, "q_len": q_len, "src": src, "cache": cache, "stride": stride,
            "block": block}


def _lens(case):
    """The request lengths of a case: listed, or spread by the case's own values."""
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    rng = random.Random("%d %d %d" % (case["reqs"], case["lo"], case["hi"]))
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["reqs"])]


def _bounds_lens(case):
    rng = random.Random("%d %d %d %d" % (case["reqs"], case["ctx_hi"], case["new_hi"], case["block"]))
    ctx = [_log(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["reqs"])]
    return ctx, new


def _shared_lens(case):
    """Requests of each group, prefix lengths, own lengths."""
    members = [int(x) for x in case["groups"].split(",")]
    prefix = [int(x) for x in case["prefix"].split(",")]
    rng = random.Random("%s %d %d" % (case["groups"], case["lo"], case["hi"]))
    return members, prefix, [_log(rng, case["lo"], case["hi"]) for _ in range(sum(members) + case["alone"])]


def _pages(length, block):
    return -(-length // block)


def _seen(length, q_len):
    """Entries that each of q_len new tokens sees of a request."""
    return [max(0, length - q_len + 1 + i) for i in range(q_len)]


def _kept(n, case):
    """Entries left of n when a token keeps its pages."""
    pages, b = _pages(n, case["block"]), case["block"]
    return n if pages <= case["keep"] else n - (pages - case["keep"]) * b


def work(case):
    op, b, s, c = case["op"], case["block"], BYTES[case["src"]], BYTES[case["cache"]]
    if op == "bounds":
        ctx, new = _bounds_lens(case)
        touched = [_pages(x + n, b) - x // b for x, n in zip(ctx, new) if n > 0]
        begun = sum(1 for x, n in zip(ctx, new) if n > 0 and x % b)
        return {"bytes": sum(new) * ENTRY * c + (sum(touched) + begun) * 2 * ENTRY * s + 4 * sum(touched) + 8 * len(ctx),
                "flops": 0}
    rows = case["heads"] * case["q_len"]
    if op == "scores":
        lens = _lens(case)
        pages = sum(_pages(n, b) for n in lens)
        width = max(1, max(_pages(n, b) for n in lens))
        return {"bytes": pages * (2 * ENTRY * s + 4) + len(lens) * (rows * (ENTRY * s + (4 if case["lse"] else 0)) + 4
                                                                     + 4 * case["q_len"] * width),
                "flops": 2 * rows * pages * ENTRY}
    if op == "sparse":
        seen = [n for x in _lens(case) for n in _seen(x, case["q_len"])]
        kept = [_kept(n, case) for n in seen]
        return {"bytes": sum(4 * _pages(n, b) for n in seen) + len(seen) * (8 * case["keep"] + 8)
                + sum(kept) * ENTRY * c + len(seen) * case["heads"] * ((ENTRY + LATENT) * s + 4),
                "flops": 2 * case["heads"] * sum(kept) * (ENTRY + LATENT)}
    members, prefix, lens = _shared_lens(case)
    keys = sum(n for m, n in zip(members, prefix) if m) + sum(lens)
    pairs = rows * (sum(m * n for m, n in zip(members, prefix)) + sum(lens))
    return {"bytes": keys * ENTRY * c + len(lens) * rows * ((ENTRY + LATENT) * s + 4) + 4 * (keys // b),
            "flops": 2 * pairs * (ENTRY + LATENT)}


# --- the inputs ------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _entries(g, blocks, block, stride, dtype):
    """A cache of N(0, 1) entries; an e4m3 one holds them divided by its scale."""
    values = torch.empty((blocks, block, stride), dtype=TYPES[dtype], device="cuda")
    step = max(1, (1 << 26) // (block * stride))
    for i in range(0, blocks, step):
        x = _normal(g, min(step, blocks - i), block, stride)
        values[i:i + step] = ((x / FP8_SCALE).clamp(-448, 448) if dtype == "fp8" else x).to(TYPES[dtype])
    return values[:, :, :ENTRY]


def _tables(g, block, *requests, spare=64):
    """Block tables of shuffled pages over one cache, one for each list of lengths (unused columns are -1), and its
    number of blocks."""
    total = sum(_pages(x, block) for lens in requests for x in lens)
    ids = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    tables, used = [], 0
    for lens in requests:
        need = torch.tensor([_pages(x, block) for x in lens], device="cuda")
        column = torch.arange(max(1, max(_pages(x, block) for x in lens)), device="cuda")
        at = used + (need.cumsum(0) - need)[:, None] + column
        table = torch.where(column < need[:, None], ids[at.clamp(max=total + spare - 1)], -1)
        tables.append(table.to(torch.int32).contiguous())
        used += sum(_pages(x, block) for x in lens)
    return tables, total + spare


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, b, src = case["op"], case["block"], TYPES[case["src"]]
    s = {"op": op, "seen": case, "block": b, "scale": torch.tensor([FP8_SCALE], device="cuda") if case["cache"] == "fp8" else None}
    if op == "bounds":
        ctx, new = _bounds_lens(case)
        (s["table"],), blocks = _tables(g, b, [x + n for x, n in zip(ctx, new)])
        s["cache"] = _entries(g, blocks, b, case["stride"], case["cache"])
        s["ctx"], s["seq_lens"] = _i32(ctx), _i32([x + n for x, n in zip(ctx, new)])
        s["span"] = max(_pages(x + n, b) - x // b for x, n in zip(ctx, new))  # pages of a request that may change
        # what is known of the pages so far: bounds of earlier entries
        middle = _normal(g, blocks, ENTRY).abs() if case["cache"] != "fp8" else _normal(g, blocks, ENTRY).abs() / FP8_SCALE
        s["bounds"] = torch.stack([middle, -middle.roll(1, 0)], 1).to(TYPES[case["cache"]]).to(src).contiguous()
        return s
    rows = (case["q_len"], case["heads"])
    if op == "scores":
        lens = _lens(case)
        (s["table"],), blocks = _tables(g, b, lens)
        s["seq_lens"] = _i32(lens)
        s["q"] = _normal(g, len(lens), *rows, ENTRY, dtype=src)
        spread = 2.3 + 0.4 * _normal(g, blocks, 2, ENTRY)  # extremes of a page of N(0, 1) values
        spread[:, 1] *= -1
        s["bounds"] = (spread / FP8_SCALE).to(TYPES["fp8"]).to(src) if case["cache"] == "fp8" else spread.to(src)
        s["lse"] = 8 + _normal(g, len(lens), *rows) if case["lse"] else None
        s["scores"] = torch.empty((len(lens), case["q_len"], s["table"].shape[1]), device="cuda")
        return s
    if op == "sparse":
        lens = _lens(case)
        (s["table"],), blocks = _tables(g, b, lens)
        tokens = len(lens) * case["q_len"]
        # page scores, of few enough values that some are equal
        s["scores"] = _normal(g, len(lens), case["q_len"], s["table"].shape[1], dtype=torch.bfloat16).float()
        s["selected"] = torch.empty((tokens, case["keep"]), dtype=torch.int32, device="cuda")
        s["selected_lens"] = torch.empty(tokens, dtype=torch.int32, device="cuda")
    else:
        members, prefix, lens = _shared_lens(case)
        (s["table"], s["prefix_table"]), blocks = _tables(g, b, lens, prefix)
        s["prefix_lens"] = _i32(prefix)
        s["cu_groups"] = _i32([sum(members[:i]) for i in range(len(members) + 1)])
        s["most"] = max(members)
    s["seq_lens"] = _i32(lens)
    s["cache"] = _entries(g, blocks, b, case["stride"], case["cache"])
    s["q"] = _normal(g, len(lens), *rows, ENTRY, dtype=src)
    s["out"] = torch.empty((len(lens), *rows, LATENT), dtype=src, device="cuda")
    s["lse"] = torch.empty((len(lens), *rows), device="cuda")
    return s


# --- one pass --------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _own_bounds(s):
    from paged_mla_kv_cache_gb300 import binding
    binding.block_bounds(s["cache"], s["bounds"], s["table"], s["seq_lens"], s["ctx"])
    return s["bounds"]


def _own_scores(s):
    from paged_mla_kv_cache_gb300 import binding
    binding.block_scores(s["q"], s["bounds"], s["table"], s["seq_lens"], s["scores"], block_size=s["block"],
                         sm_scale=SCALE, scale=s["scale"], lse=s["lse"])
    return s["scores"]


def _own_sparse(s):
    from paged_mla_kv_cache_gb300 import binding
    if "workspace" not in s:  # kept by a serving loop
        s["workspace"] = binding.new_attention_workspace("cuda")
    case, q, out = s["seen"], s["q"], s["out"]
    binding.select_blocks(s["scores"], s["table"], s["seq_lens"], s["selected"], s["selected_lens"],
                          block_size=s["block"], first=case["first"], last=case["last"])
    # every token is a request of its own over its pages
    binding.latent_decode(q.view(-1, 1, *q.shape[2:]), s["cache"], s["selected"], s["selected_lens"],
                          out.view(-1, 1, *out.shape[2:]), s["lse"], sm_scale=SCALE, scale=s["scale"],
                          workspace=s["workspace"])
    return [s["selected"], s["selected_lens"], out, s["lse"]]


def _own_shared(s):
    from paged_mla_kv_cache_gb300 import binding
    if "workspace" not in s:
        s["workspace"] = binding.new_shared_workspace("cuda", *s["out"].shape)
    binding.latent_decode_shared(s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["cu_groups"], s["table"],
                                 s["seq_lens"], s["out"], s["lse"], sm_scale=SCALE, scale=s["scale"],
                                 workspace=s["workspace"])
    return [s["out"], s["lse"]]


def _plain_bounds(s):
    b, ctx, end = s["block"], s["ctx"].long(), s["seq_lens"].long()
    page = (ctx // b)[:, None] + torch.arange(s["span"], device=ctx.device)                 # [reqs, span]
    place = page[:, :, None] * b + torch.arange(b, device=ctx.device)
    joins = (place >= ctx[:, None, None]) & (place < end[:, None, None])
    touched = joins.any(-1)
    ids = s["table"].gather(1, page.clamp(max=s["table"].shape[1] - 1))[touched].long()
    entries, joins = s["cache"][ids].float(), joins[touched][:, :, None]
    hi = torch.where(joins, entries, -math.inf).amax(1)
    lo = torch.where(joins, entries, math.inf).amin(1)
    begun = (page * b < ctx[:, None])[touched][:, None]
    before = s["bounds"][ids].float()
    hi = torch.where(begun, torch.maximum(hi, before[:, 0]), hi)
    lo = torch.where(begun, torch.minimum(lo, before[:, 1]), lo)
    s["bounds"][ids] = torch.stack([hi, lo], 1).to(s["bounds"].dtype)
    return s["bounds"]


def _limits(s, q_len):
    """Entries that each token of each request sees."""
    lens = s["seq_lens"][:, None] - q_len + 1 + torch.arange(q_len, device=s["seq_lens"].device)
    return lens.clamp(min=0)


def _plain_scores(s):
    q, b = s["q"].float(), s["block"]
    n, q_len, h, _ = q.shape
    pages = s["bounds"][s["table"].clamp(min=0).long()].float()                              # [reqs, width, 2, ENTRY]
    if s["scale"] is not None:
        pages = pages * s["scale"]
    rows = q.view(n, q_len * h, ENTRY)
    x = torch.bmm(rows.clamp(min=0), pages[:, :, 0].transpose(1, 2)) + torch.bmm(rows.clamp(max=0), pages[:, :, 1].transpose(1, 2))
    x = (x * SCALE).view(n, q_len, h, -1)
    if s["lse"] is not None:
        x = x - s["lse"][..., None]
    column = torch.arange(pages.shape[1], device=q.device)
    return torch.where(column * b < _limits(s, q_len)[..., None], x.amax(2), -math.inf)


def _attend(scores, seen, values):
    """Softmax over the last axis where `seen`; rows that see nothing give 0 and a log sum of -inf."""
    scores = torch.where(seen, scores, -math.inf)
    most = scores.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    p = torch.exp(scores - most)
    total = p.sum(-1, keepdim=True)
    out = values(p) / torch.where(total == 0, 1.0, total)
    return out, (most + torch.log(total)).squeeze(-1)


def _latent(q, s, table, lens):
    """Rows [n, rows, ENTRY] over the entries of their table; `lens` [n, rows] of them are seen."""
    kv = s["cache"][table.clamp(min=0).long()].reshape(len(table), -1, ENTRY).float()
    if s["scale"] is not None:
        kv = kv * s["scale"]
    seen = torch.arange(kv.shape[1], device=q.device) < lens[..., None]
    return _attend(torch.bmm(q, kv.transpose(1, 2)) * SCALE, seen, lambda p: torch.bmm(p, kv[:, :, :LATENT]))


def _plain_sparse(s):
    case, b = s["seen"], s["block"]
    keep, first, last = case["keep"], case["first"], case["last"]
    n, q_len, h, _ = s["q"].shape
    table = s["table"].repeat_interleave(q_len, 0)
    seen = _limits(s, q_len).view(-1, 1)
    pages = (seen + b - 1) // b
    column = torch.arange(table.shape[1], device=table.device)
    free = (column >= first) & (column < pages - last)                                       # pages that compete
    order = torch.where(free, s["scores"].view(n * q_len, -1), -math.inf).sort(dim=1, descending=True, stable=True)[1]
    rank = order.argsort(1)
    chosen = (column < pages) & (~free | (rank < keep - first - last) | (pages <= keep))
    place = torch.where(chosen, column, table.shape[1]).sort(1)[0]
    place = torch.nn.functional.pad(place, (0, max(0, keep - place.shape[1])), value=table.shape[1])[:, :keep]
    selected = torch.where(place < table.shape[1], table.gather(1, place.clamp(max=table.shape[1] - 1)), -1)
    lens = torch.where(pages <= keep, seen, seen - (pages - keep) * b).int()
    out, lse = _latent(s["q"].float().view(n * q_len, h, ENTRY), s, selected, lens.expand(-1, h))
    return [selected, lens.view(-1), out.view(s["out"].shape).to(s["out"].dtype), lse.view(n, q_len, h)]


def _plain_shared(s):
    q = s["q"].float()
    n, q_len, h, _ = q.shape
    out, lse = _latent(q.view(n, q_len * h, ENTRY), s, s["table"], _limits(s, q_len).repeat_interleave(h, 1))
    # the rows of each group side by side, padded to the largest group
    cu = s["cu_groups"].long()
    member = torch.arange(max(1, s["most"]), device=q.device)
    at = (cu[:-1, None] + member)
    real = at < cu[1:, None]
    rows = q[at.clamp(max=n - 1)].view(len(at), -1, ENTRY)
    lens = torch.where(real, s["prefix_lens"][:, None], 0).repeat_interleave(q_len * h, 1)
    prev, prev_lse = _latent(rows, s, s["prefix_table"], lens)
    all_prev, all_lse = torch.zeros_like(out), torch.full_like(lse, -math.inf)
    all_prev[at[real]] = prev.view(*at.shape, q_len * h, LATENT)[real]
    all_lse[at[real]] = prev_lse.view(*at.shape, q_len * h)[real]
    both = torch.logaddexp(lse, all_lse)
    base = torch.where(both == -math.inf, 0.0, both)
    out = out * torch.exp(lse - base)[..., None] + all_prev * torch.exp(all_lse - base)[..., None]
    return [out.view(s["out"].shape).to(s["out"].dtype), both.view(n, q_len, h)]


_run_own = {"bounds": _own_bounds, "scores": _own_scores, "sparse": _own_sparse, "shared": _own_shared}
_run_plain = {"bounds": _plain_bounds, "scores": _plain_scores, "sparse": _plain_sparse, "shared": _plain_shared}


# --- the definition in 64 bits ------------------------------------------------------

def _exact_rows(q, kv):
    """Queries [rows, ENTRY] over entries [n, ENTRY], all of them seen, in 64 bits."""
    if len(kv) == 0:
        return q.new_zeros((len(q), LATENT)), q.new_full((len(q),), -math.inf)
    x = q @ kv.T * SCALE
    z = torch.logsumexp(x, 1)
    return torch.exp(x - z[:, None]) @ kv[:, :LATENT], z


def exact(case, seed):
    op, b = case["op"], case["block"]
    s = prepare(case, seed)
    factor = 1.0 if s["scale"] is None else s["scale"].double()
    if op == "bounds":
        bounds = s["bounds"].double()
        ctx, new = _bounds_lens(case)
        for r, (x, n) in enumerate(zip(ctx, new)):
            if n == 0:
                continue
            pages = s["table"][r, x // b:_pages(x + n, b)].long()
            kv = s["cache"][pages].double().flatten(0, 1)[x % b:x % b + n]
            kv = torch.nn.functional.pad(kv, (0, 0, x % b, len(pages) * b - x % b - n), value=math.nan).view(-1, b, ENTRY)
            hi, lo = kv.nan_to_num(nan=-math.inf).amax(1), kv.nan_to_num(nan=math.inf).amin(1)
            if x % b:
                hi[0], lo[0] = torch.maximum(hi[0], bounds[pages[0], 0]), torch.minimum(lo[0], bounds[pages[0], 1])
            bounds[pages] = torch.stack([hi, lo], 1)
        return bounds
    if op == "scores":
        scores = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for r, n in enumerate(_lens(case)):
            for i, seen in enumerate(_seen(n, case["q_len"])):
                pages = s["table"][r, :_pages(seen, b)].long()
                if len(pages) == 0:
                    continue
                q, page = s["q"][r, i].double()[:, None], s["bounds"][pages].double() * factor
                step = max(1, (1 << 27) // (len(pages) * ENTRY))
                x = torch.cat([torch.maximum(q[h:h + step] * page[:, 0], q[h:h + step] * page[:, 1]).sum(-1)
                               for h in range(0, len(q), step)]) * SCALE
                if s["lse"] is not None:
                    x = x - s["lse"][r, i].double()[:, None]
                scores[r, i, :len(pages)] = x.amax(0)
        return scores
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")

    def entries(ids, n):
        return s["cache"][ids.long()].reshape(-1, ENTRY)[:n].double() * factor

    if op == "sparse":
        for r, n in enumerate(_lens(case)):
            for i, seen in enumerate(_seen(n, case["q_len"])):
                pages = list(range(_pages(seen, b)))
                if len(pages) > case["keep"]:
                    score = s["scores"][r, i].tolist()
                    ends = pages[:case["first"]] + pages[len(pages) - case["last"]:]
                    best = sorted(pages[case["first"]:len(pages) - case["last"]], key=lambda c: (-score[c], c))
                    pages = sorted(ends + best[:case["keep"] - len(ends)])
                kv = entries(s["table"][r][pages], _kept(seen, case))
                out[r, i], lse[r, i] = _exact_rows(s["q"][r, i].double(), kv)
        return [None, None, out, lse]
    members, prefix, lens = _shared_lens(case)
    group = [g for g, m in enumerate(members) for _ in range(m)]
    known, before = None, None
    for r, n in enumerate(lens):
        if r < len(group) and known != group[r]:
            known = group[r]
            before = entries(s["prefix_table"][known, :_pages(prefix[known], b)], prefix[known])
        mine = entries(s["table"][r, :_pages(n, b)], n)
        for i, seen in enumerate(_seen(n, case["q_len"])):
            kv = torch.cat([before, mine[:seen]]) if r < len(group) else mine[:seen]
            out[r, i], lse[r, i] = _exact_rows(s["q"][r, i].double(), kv)
    return [out, lse]

"""Plain 64-bit definitions of the operators for long contexts. Loops over
requests and pages; nothing of the framework."""
import math

import torch

from mla_reference import attend


def bounds(cache, before, table, seq, ctx=None):
    """What `before` [blocks, 2, E] becomes, in its type."""
    got = before.clone()
    blocks, B, _ = cache.shape
    for r in range(len(seq)):
        a, b = max(int(ctx[r]), 0) if ctx is not None else 0, max(int(seq[r]), 0)
        b = min(b, table.shape[1] * B)
        if b <= a:
            continue
        for c in range(a // B, -(-b // B)):
            ident = int(table[r, c])
            if not 0 <= ident < blocks:
                continue
            rows = cache[ident, max(a - c * B, 0):min(b - c * B, B)].double()
            hi, lo = rows.amax(0), rows.amin(0)
            if c * B < a:
                hi, lo = torch.maximum(hi, before[ident, 0].double()), torch.minimum(lo, before[ident, 1].double())
            got[ident, 0], got[ident, 1] = hi.to(got.dtype), lo.to(got.dtype)
    return got


def seen(length, i, q_len, room):
    return min(max(max(int(length), 0) - q_len + 1 + i, 0), room)


def scores(q, bound, table, seq, block_size, factor, lse=None):
    """Scores [R, n, W] and what bounds their errors: the largest sum |q b| factor + |lse| of a head."""
    R, n, H, E = q.shape
    W = table.shape[1]
    out = torch.full((R, n, W), -math.inf, dtype=torch.float64, device=q.device)
    mag = torch.zeros(R, n, W, dtype=torch.float64, device=q.device)
    for r in range(R):
        for i in range(n):
            for c in range(-(-seen(seq[r], i, n, W * block_size) // block_size)):
                ident = int(table[r, c])
                if not 0 <= ident < bound.shape[0]:
                    continue
                x, (hi, lo) = q[r, i].double(), bound[ident].double()
                terms = torch.where(x < 0, x * lo, x * hi)
                shift = torch.zeros(H, dtype=torch.float64, device=q.device)
                if lse is not None:
                    shift = torch.where(lse[r, i].isfinite(), lse[r, i].double(), 0.0)
                s = terms.sum(1) * factor - shift
                out[r, i, c] = s.max() if not s.isnan().any() else math.nan
                mag[r, i, c] = (terms.abs().sum(1) * factor + shift.abs()).max()
    return out, mag


def select(score, table, seq, q_len, block_size, keep, first, last):
    """Lists: ids and columns of each token's pages (-1 behind the last), and entries on them."""
    ids, columns, lens = [], [], []
    R, W = len(table), len(table[0]) if len(table) else 0
    for r in range(R):
        for i in range(q_len):
            n = seen(seq[r], i, q_len, W * block_size)
            pages = list(range(-(-n // block_size)))
            kept, m = pages, n
            if len(pages) > keep:
                ends = pages[:first] + pages[len(pages) - last:]
                # NaN above all, then the largest, then the lowest column
                rank = sorted(pages[first:len(pages) - last],
                              key=lambda c: (0, 0.0, c) if math.isnan(score[r][i][c]) else (1, -score[r][i][c], c))
                kept = sorted(ends + rank[:keep - first - last])
                m = n - (len(pages) - keep) * block_size
            fill = [-1] * (keep - len(kept))
            ids.append([int(table[r][c]) for c in kept] + fill)
            columns.append(kept + fill)
            lens.append(m)
    return ids, columns, lens


def _entries(cache, row, length, factor):
    """Entries of a table's row, in 64 bits, and which of them are there."""
    B = cache.shape[1]
    m = min(max(int(length), 0), len(row) * B)
    pages = row[:-(-m // B)].long()
    good = (pages >= 0) & (pages < cache.shape[0])
    kv = cache[torch.where(good, pages, 0)].reshape(-1, cache.shape[2])[:m].double() * factor
    ok = good.repeat_interleave(B)[:m]
    return torch.where(ok[:, None], kv, 0.0), ok


def shared(q, cache, prefix_table, prefix_lens, cu, table, lens, dv, sm_scale, factor=1.0):
    """As mla_reference.decode, the entries of a request's group before its own."""
    R, n, H, E = q.shape
    out = torch.zeros(R, n, H, dv, dtype=torch.float64, device=q.device)
    lse = torch.full((R, n, H), -math.inf, dtype=torch.float64, device=q.device)
    pv, worst, flat = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(out)
    # (requests before the first boundary have no prefix, whatever later boundaries say)
    group = {r: g for g in range(len(cu) - 1) for r in range(max(int(cu[0]), int(cu[g]), 0), min(max(int(cu[g + 1]), 0), R))}
    none = torch.zeros(0, dtype=torch.int32, device=q.device)
    for r in range(R):
        g = group.get(r)
        before, ok0 = _entries(cache, none, 0, factor) if g is None else _entries(cache, prefix_table[g], prefix_lens[g], factor)
        mine, ok1 = _entries(cache, table[r], lens[r], factor)
        place = torch.arange(len(mine), device=q.device)
        for i in range(n):
            see = torch.cat([ok0, ok1 & (place < max(int(lens[r]), 0) - n + 1 + i)])
            if len(see) == 0:
                continue
            kv = torch.cat([before, mine])
            out[r, i], lse[r, i], pv[r, i], worst[r, i], flat[r, i] = attend(
                q[r, i].double(), kv, kv[:, :dv], see[None].expand(H, len(see)), sm_scale)
    return out, lse, pv, worst, flat

"""Plain 64-bit definitions of the operators around the gather, and the error
bounds their tests use. Loops over requests; nothing of the framework.

A rounding to type t is off by at most u(t) = eps(t) / 2 of the value. Sums of n
terms in 32 bits are off by at most n * 2^-24 of the sum of magnitudes (the
tensor cores may cut instead of round, 2^-23 for each of the n / 16 additions of
a group of products: less)."""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


def plan(ctx, new, table, free, block_size, num_blocks, max_tokens):
    """Lists of Python whole numbers, token by token and page by page."""
    table = [list(map(int, row)) for row in table]
    slots, positions, seqs, cu_new, cu_seq, lens, used = [], [], [], [0], [0], [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        for page in range(-(-c // block_size), -(-(c + n) // block_size)):
            ident = int(free[used]) if used < len(free) else -1
            ident = ident if 0 <= ident < num_blocks else -1
            used += 1
            if page < len(table[r]):
                table[r][page] = ident
        for p in range(c, c + n):
            page = p // block_size
            ident = table[r][page] if page < len(table[r]) else -1
            slots.append(ident * block_size + p % block_size if 0 <= ident < num_blocks else -1)
            positions.append(p)
            seqs.append(r)
        lens.append(c + n)
        cu_new.append(cu_new[-1] + n)
        cu_seq.append(cu_seq[-1] + c + n)
    fill = max(0, max_tokens - len(slots))
    tail = [-1] * fill
    return (table, (slots + tail)[:max_tokens], (positions + tail)[:max_tokens], (seqs + tail)[:max_tokens], cu_new,
            lens, cu_seq, min(used, len(free)))


def rotate(x, cs, pairs):
    """x [n, ..., d] and cs [n, d] in 64 bits; the rotation and the sum of magnitudes of each element."""
    half = x.shape[-1] // 2
    cs = cs.view(cs.shape[0], *([1] * (x.dim() - 2)), 2 * half)
    cos, sin = cs[..., :half], cs[..., half:]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :half], x[..., half:])
    out = [a * cos - b * sin, b * cos + a * sin]
    mag = [(a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()]
    join = (lambda y: torch.stack(y, -1).flatten(-2)) if pairs else (lambda y: torch.cat(y, -1))
    return join(out), join(mag)


def attend(q, k, v, seen, sm_scale):
    """One head group: q [n, e], k [m, e], v [m, d], seen [n, m], all 64 bits. Returns out, lse, and what bounds the
    errors: sum p|v|, the largest sum |q k| sm_scale of a seen key, and the largest p times sum |v| of seen keys."""
    s = q @ k.T * sm_scale
    mag = (q.abs() @ k.abs().T * sm_scale).masked_fill(~seen, 0.0)
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, 1) if s.shape[1] else torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    worst = mag.amax(1) if mag.shape[1] else torch.zeros_like(lse)
    v = torch.where(seen.any(0)[:, None], v, 0.0)
    flat = (p.amax(1)[:, None] if p.shape[1] else 0.0) * (seen.double() @ v.abs())
    return p @ v, lse, p @ v.abs(), worst, flat


def decode(q, cache, table, lens, dv, sm_scale, factor=1.0):
    """q [R, n, H, E]; cache [blocks, B, E]. Entries of pages outside the cache or the table are left out."""
    R, n, H, E = q.shape
    B = cache.shape[1]
    out = torch.zeros(R, n, H, dv, dtype=torch.float64, device=q.device)
    lse = torch.full((R, n, H), -math.inf, dtype=torch.float64, device=q.device)
    pv, worst, flat = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(out)
    for r in range(R):
        length = max(int(lens[r]), 0)
        m = min(length, table.shape[1] * B)
        if m == 0:
            continue
        pages = table[r, :-(-m // B)].long()
        good = (pages >= 0) & (pages < cache.shape[0])
        kv = cache[torch.where(good, pages, 0)].reshape(-1, E)[:m].double() * factor
        ok = good.repeat_interleave(B)[:m]
        kv = torch.where(ok[:, None], kv, 0.0)
        place = torch.arange(m, device=q.device)
        for i in range(n):
            seen = (ok & (place < length - n + 1 + i))[None].expand(H, m)
            out[r, i], lse[r, i], pv[r, i], worst[r, i], flat[r, i] = attend(q[r, i].double(), kv, kv[:, :dv], seen,
                                                                             sm_scale)
    return out, lse, pv, worst, flat


def prefill(q, k, pe, v, cu_q, cu_k, sm_scale, causal, prev_out=None, prev_lse=None):
    tq, H, _ = q.shape
    out = torch.zeros(tq, H, v.shape[2], dtype=torch.float64, device=q.device)
    lse = torch.full((tq, H), -math.inf, dtype=torch.float64, device=q.device)
    pv, worst = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(cu_q) - 1):
        a, b, c, d = int(cu_q[r]), int(cu_q[r + 1]), int(cu_k[r]), int(cu_k[r + 1])
        if b <= a or d <= c:
            continue
        seen = torch.ones(b - a, d - c, dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril((d - c) - (b - a))
        for h in range(H):
            key = torch.cat([k[c:d, h], pe[c:d]], 1).double()
            out[a:b, h], lse[a:b, h], pv[a:b, h], worst[a:b, h], _ = attend(q[a:b, h].double(), key,
                                                                          v[c:d, h].double(), seen, sm_scale)
    if prev_lse is not None:
        both = torch.logaddexp(lse, prev_lse.double())
        x = torch.where(both == -math.inf, 0.0, both)
        w0, w1 = torch.exp(lse - x)[..., None], torch.exp(prev_lse.double() - x)[..., None]
        prev = torch.where(w1 == 0, 0.0, prev_out.double())
        out, pv, lse = out * w0 + prev * w1, pv * w0 + prev.abs() * w1, both
    return out, lse, pv, worst


def check_attention(got, got_lse, want, want_lse, pv, worst, entry, weights_u, extra=0.0, weights_abs=0.0):
    """Scores are sums of `entry` products in 32 bits (`extra`: a further bound on them), so each weight is off by a
    factor within exp(2 ds); weights are rounded with unit weights_u for the second product (weights_abs: and by a step
    below it, already times the magnitudes it meets), sums of values in 32 bits
    (2^-18 of the magnitudes covers 64 additions in a row), and the result is rounded to its own type."""
    ds = (entry + 64) * 2.0 ** -24 * worst + extra
    finite = want_lse != -math.inf
    assert torch.equal(got_lse[~finite], want_lse[~finite].float())
    err = (got_lse.double() - want_lse).abs()[finite]
    bound = (ds + 2.0 ** -20 * (4 + want_lse.abs()))[finite]
    assert (err <= bound).all(), f"lse off by {err.max():.3g}, {(err / bound).max():.3g} of its bound"
    err = (got.double() - want).abs()
    bound = U[got.dtype] * want.abs() + (2 * ds[..., None] + weights_u + 2.0 ** -18) * pv * 1.01 + weights_abs + 1e-30
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25
    assert not got.isnan().any(), "NaN"
    assert (err <= bound).all(), f"out off by {err.max():.3g}, {(err / bound).max():.3g} of its bound"


def tables(rng, lens, block_size, spare=3):
    """Block ids of shuffled pages of requests of these lengths; unused columns are -1. Returns table, number of blocks."""
    need = [-(-max(x, 0) // block_size) for x in lens]
    ids = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(max(need, default=0), 1)), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, len(ids)

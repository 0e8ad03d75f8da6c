"""Serving steps of one latent-attention layer over the paged cache.

The operators together, as a serving loop uses them: plan_step lays out the
step's pages and slots, append norms, rotates and writes the new entries, and
the attention runs either absorbed over the paged cache (latent_decode, one or
a few new tokens a request) or expanded (latent_prefill: the chunk's own keys,
causal, then the gathered context in pieces, joined by their states).

    python examples/serve_step.py            # a few requests on cuda:0

Weights are random; projections are plain torch products.
"""
from __future__ import annotations

import dataclasses
import math
import os
import sys
from typing import List, Optional

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_mla_kv_cache_gb300 import binding  # noqa: E402


@dataclasses.dataclass
class LayerConfig:
    hidden: int = 256
    heads: int = 16
    latent: int = 512
    rope: int = 64
    nope: int = 128
    value: int = 128
    block_size: int = 64
    max_positions: int = 4096
    eps: float = 1e-6


class LatentLayer:
    """One attention layer with its paged cache and the buffers of its steps."""

    def __init__(self, cfg: LayerConfig, num_blocks: int, max_reqs: int, max_tokens: int, dtype=torch.bfloat16,
                 cache_dtype=None, cache_scale: Optional[float] = None, device="cuda:0", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) / math.sqrt(shape[0])).to(dtype)

        self.cfg, self.dtype, self.device = cfg, dtype, device
        c = cfg
        self.w_q = weight(c.hidden, c.heads * (c.nope + c.rope))
        self.w_down = weight(c.hidden, c.latent + c.rope)
        self.w_up = weight(c.latent, c.heads * (c.nope + c.value))  # keys and values of every head, side by side
        self.norm = torch.ones(c.latent, device=device)
        angle = torch.arange(c.max_positions, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(c.rope // 2, dtype=torch.float64) / (c.rope // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.cache = torch.zeros(num_blocks, c.block_size, c.latent + c.rope, device=device).to(cache_dtype or dtype)
        self.scale = None if cache_scale is None else torch.tensor([cache_scale], device=device)
        self.sm_scale = 1.0 / math.sqrt(c.nope + c.rope)

        # a serving loop's state: pages of every request, lengths, the ids that are free
        i32 = dict(dtype=torch.int32, device=device)
        width = -(-c.max_positions // c.block_size)
        self.table = torch.full((max_reqs, width), -1, **i32)
        self.lens = torch.zeros(max_reqs, **i32)
        self.free = torch.randperm(num_blocks, generator=g, device=device).to(torch.int32)
        self.slots = torch.empty(max_tokens, dtype=torch.int64, device=device)
        self.positions = torch.empty(max_tokens, **i32)
        self.token_to_seq = torch.empty(max_tokens, **i32)
        self.cu_new, self.cu_seq = torch.empty(max_reqs + 1, **i32), torch.empty(max_reqs + 1, **i32)
        self.taken = torch.zeros(1, **i32)
        self.error = torch.zeros(1, **i32)
        self.gather_ws = binding.new_workspace(device)
        self.attention_ws = binding.new_attention_workspace(device)

    # -- what every step begins with

    def begin(self, hidden: torch.Tensor, new_lens: List[int]):
        """Pages and slots for the new tokens, their entries in the cache, their queries rotated. Returns the queries
        [tokens, heads, nope + rope] and the lengths before the step."""
        c, n = self.cfg, hidden.shape[0]
        new = torch.tensor(new_lens, dtype=torch.int32, device=self.device)
        before = self.lens.clone()
        after = torch.empty_like(self.lens)
        binding.plan_step(before, new, self.table, self.free, c.block_size, self.slots[:n], self.positions[:n],
                          self.token_to_seq[:n], self.cu_new, after, self.cu_seq, self.taken, self.cache.shape[0],
                          self.error)
        q = (hidden @ self.w_q).view(n, c.heads, c.nope + c.rope)
        down = hidden @ self.w_down
        q_pe = q[:, :, c.nope:]
        binding.append(down[:, :c.latent], down[:, c.latent:], self.cache, self.slots[:n], self.positions[:n],
                       self.cos_sin, norm_weight=self.norm, eps=c.eps, scale=self.scale, q_pe=q_pe, q_out=q_pe,
                       interleaved=True, error_flag=self.error)
        self.lens = after
        self.free = self.free[int(self.taken):]  # a serving engine keeps the count on the host, one step behind
        return q, before

    # -- absorbed: a few new tokens a request

    def decode(self, hidden: torch.Tensor, q_len: int = 1) -> torch.Tensor:
        """q_len new tokens for every request; returns [tokens, heads, value]."""
        c, r = self.cfg, self.lens.shape[0]
        q, _ = self.begin(hidden, [q_len] * r)
        up = self.w_up.view(c.latent, c.heads, c.nope + c.value)
        # keys' up-projection moves to the queries, values' to the result
        absorbed = torch.empty(r, q_len, c.heads, c.latent + c.rope, dtype=self.dtype, device=self.device)
        absorbed[..., :c.latent] = torch.einsum("thn,lhn->thl", q[:, :, :c.nope], up[:, :, :c.nope]).view(
            r, q_len, c.heads, c.latent)
        absorbed[..., c.latent:] = q[:, :, c.nope:].view(r, q_len, c.heads, c.rope)
        out = torch.empty(r, q_len, c.heads, c.latent, dtype=self.dtype, device=self.device)
        binding.latent_decode(absorbed, self.cache, self.table, self.lens, out, sm_scale=self.sm_scale, scale=self.scale,
                              workspace=self.attention_ws, error_flag=self.error)
        return torch.einsum("rqhl,lhv->rqhv", out, up[:, :, c.nope:]).reshape(-1, c.heads, c.value)

    # -- expanded: a chunk of new tokens over its own keys and the cached context

    def prefill(self, hidden: torch.Tensor, new_lens: List[int], chunk: int = 1024) -> torch.Tensor:
        """new_lens[r] new tokens for request r; returns [tokens, heads, value]. The cached context is gathered,
        expanded and attended in pieces of `chunk` tokens a request."""
        c, n = self.cfg, hidden.shape[0]
        q, before = self.begin(hidden, new_lens)
        out = torch.empty(n, c.heads, c.value, dtype=self.dtype, device=self.device)
        lse = torch.empty(n, c.heads, device=self.device)

        def attend(starts: torch.Tensor, lens: torch.Tensor, causal: bool, joined: bool):
            cu = torch.cat([lens.new_zeros(1), lens.cumsum(0, dtype=torch.int32)])
            total = int(cu[-1])
            entries = torch.empty(total, c.latent + c.rope, dtype=self.dtype, device=self.device)
            binding.gather(self.cache, entries, self.table, cu, starts, self.scale, self.error, workspace=self.gather_ws)
            up = (entries[:, :c.latent] @ self.w_up).view(total, c.heads, c.nope + c.value)
            binding.latent_prefill(q, up[:, :, :c.nope], entries[:, c.latent:], up[:, :, c.nope:], self.cu_new, cu, out,
                                   lse, sm_scale=self.sm_scale, causal=causal, prev_out=out if joined else None,
                                   prev_lse=lse if joined else None, workspace=self.attention_ws, error_flag=self.error)

        attend(before, torch.tensor(new_lens, dtype=torch.int32, device=self.device), True, False)
        for start in range(0, int(before.max()), chunk):
            attend(torch.full_like(before, start).minimum(before), (before - start).clamp(0, chunk), False, True)
        return out


def main():
    torch.manual_seed(0)
    layer = LatentLayer(LayerConfig(), num_blocks=64, max_reqs=3, max_tokens=512)
    prompt = [200, 3, 65]
    x = torch.randn(sum(prompt), layer.cfg.hidden, device="cuda").bfloat16()
    print("prefill", tuple(layer.prefill(x, prompt).shape), "lengths", layer.lens.tolist())
    x = torch.randn(100, layer.cfg.hidden, device="cuda").bfloat16()
    print("next chunk", tuple(layer.prefill(x, [0, 90, 10], chunk=64).shape), "lengths", layer.lens.tolist())
    for _ in range(3):
        x = torch.randn(3, layer.cfg.hidden, device="cuda").bfloat16()
        y = layer.decode(x)
    print("decode", tuple(y.shape), "lengths", layer.lens.tolist(), "error flag", int(layer.error))


if __name__ == "__main__":
    main()

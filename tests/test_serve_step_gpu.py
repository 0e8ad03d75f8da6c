"""The serving example: its two attention paths against each other and against the formula in 64 bits."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    return cuda_lib


def rotate(x, positions, rope):
    """Neighbours turned by the position's angles, in 64 bits."""
    half = rope // 2
    angle = positions.double()[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    turn = torch.polar(torch.ones_like(angle), angle)
    z = torch.view_as_complex(x.double().unflatten(-1, (half, 2)).contiguous())
    z = z * (turn if x.dim() == 2 else turn[:, None])
    return torch.view_as_real(z).flatten(-2)


def expected(layer, tokens, new):
    """Attention of the last `new` of `tokens` [n, hidden] of one request, expanded, in 64 bits from the same 16-bit
    weights, entries rounded to the cache's type as append stores them."""
    c = layer.cfg
    n = tokens.shape[0]
    pos = torch.arange(n, device=tokens.device)
    down = (tokens @ layer.w_down).double()
    latent = down[:, :c.latent]
    latent = latent / (latent.square().mean(1, keepdim=True) + c.eps).sqrt()
    entry = torch.cat([latent, rotate(down[:, c.latent:], pos, c.rope)], 1).to(layer.dtype).double()
    up = (entry[:, :c.latent] @ layer.w_up.double()).view(n, c.heads, c.nope + c.value)
    q = (tokens @ layer.w_q).view(n, c.heads, -1)[-new:]
    qr = rotate(q[:, :, c.nope:], pos[-new:], c.rope)
    s = torch.einsum("qhd,khd->hqk", q[:, :, :c.nope].double(), up[:, :, :c.nope])
    s = (s + torch.einsum("qhd,kd->hqk", qr, entry[:, c.latent:])) * layer.sm_scale
    s = s.masked_fill(torch.ones(new, n, dtype=torch.bool, device=s.device).triu(n - new + 1), float("-inf"))
    return torch.einsum("hqk,khv->qhv", s.softmax(2), up[:, :, c.nope:])


def test_steps_match_the_formula():
    from serve_step import LatentLayer, LayerConfig
    torch.manual_seed(3)
    cfg = LayerConfig(heads=4)
    layer = LatentLayer(cfg, num_blocks=40, max_reqs=3, max_tokens=600)
    hist = [torch.zeros(0, cfg.hidden, device="cuda", dtype=torch.bfloat16) for _ in range(3)]

    def step(lens, run):
        x = torch.randn(sum(lens), cfg.hidden, device="cuda").bfloat16()
        parts = x.split(lens)
        out = run(x).split(lens)
        for r in range(3):
            hist[r] = torch.cat([hist[r], parts[r]])
            if lens[r] == 0:
                continue
            want = expected(layer, hist[r], lens[r])
            # values and the few roundings between (projections, weights, results) to 8 bits: each 2^-8 of magnitudes of
            # about the values' own, which is 3 at most here
            assert (out[r].double() - want).abs().max() < 12 * 2.0 ** -8 * want.abs().max().clamp(min=1.0)
        assert layer.lens.tolist() == [h.shape[0] for h in hist] and int(layer.error) == 0

    step([200, 3, 65], lambda x: layer.prefill(x, [200, 3, 65]))
    step([0, 90, 10], lambda x: layer.prefill(x, [0, 90, 10], chunk=64))
    for _ in range(2):
        step([1, 1, 1], layer.decode)
    step([2, 2, 2], lambda x: layer.decode(x, q_len=2))


def test_fp8_cache_runs_and_stays_near():
    from serve_step import LatentLayer, LayerConfig
    torch.manual_seed(4)
    cfg = LayerConfig(heads=4)
    a = LatentLayer(cfg, num_blocks=16, max_reqs=2, max_tokens=300)
    b = LatentLayer(cfg, num_blocks=16, max_reqs=2, max_tokens=300, cache_dtype=torch.float8_e4m3fn, cache_scale=0.02)
    x = torch.randn(170, cfg.hidden, device="cuda").bfloat16()
    y = torch.randn(2, cfg.hidden, device="cuda").bfloat16()
    pa, pb = a.prefill(x, [150, 20]), b.prefill(x, [150, 20])
    da, db = a.decode(y), b.decode(y)
    assert int(b.error) == 0
    # entries of 4 significant bits: off by 2^-4 at most, by about 2^-5.5 in the mean, here averaged further
    for u, v in ((pa, pb), (da, db)):
        assert (u.float() - v.float()).norm() < 0.15 * u.float().norm()

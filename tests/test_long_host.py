"""Refusals of the operators for long contexts, on the host, before any CUDA call."""
import os
import re
import subprocess

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding, build

import test_mla_devices_host as devices
from test_mla_devices_host import F32, I32, launches, placed  # noqa: F401  (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_the_operators(cuda_lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pmg_long.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(pmg_\w+)\s*\(", text, flags=re.M)))
    assert names == ["pmg_block_bounds", "pmg_block_scores", "pmg_latent_decode_shared", "pmg_select_blocks",
                     "pmg_shared_workspace"]
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB_PATH], capture_output=True, text=True, check=True)
    for name in names:
        assert re.search(rf"\bT {name}$", out.stdout, flags=re.M)
    assert [int(x) for x in re.findall(r"#define PMG_CALL_\w+ (\d+)", text)] == [4, 5, 6, 7]


# The arguments of each call, in order, of a call that would run; what a value in place of one makes of it.
BOUNDS = dict(cache=4096, blk=64 * 576, tok=576, nb=4, B=64, E=576, cdt=0, bounds=4096, bb=1152, br=576, bdt=0, bt=4096, bts=4,
              ctx=4096, seq=4096, R=2, err=4096, stream=0)
SCORES = dict(q=4096, qr=576, qt=576, qh=576, bounds=4096, bb=1152, br=576, nb=4, bt=4096, bts=4, seq=4096, R=2, n=1, H=1, E=576,
              B=64, dt=0, scale=4096, sm=0.1, lse=4096, scores=4096, ss=4, err=4096, stream=0, opt=0)
SELECT = dict(scores=4096, ss=4, bt=4096, bts=4, seq=4096, R=2, n=1, B=64, sel=4096, sels=3, cols=4096, lens=4096, keep=3,
              first=1, last=1, err=4096, stream=0)
SHARED = dict(q=4096, qr=576, qt=576, qh=576, cache=4096, bs=64 * 576, ts=576, nb=4, pt=4096, pts=4, pl=4096, cu=4096, G=1, bt=4096,
              bts=4, lens=4096, R=2, n=1, H=1, dv=512, dr=64, B=64, qdt=0, cdt=0, scale=4096, sm=0.1, out=4096, orr=512, ot=512,
              oh=512, lse=4096, ws=4096, wsb=0, err=4096, stream=0, opt=0)
BIG = 2 ** 41


@pytest.mark.parametrize("over,status", [
    (dict(cache=0), 1), (dict(bounds=0), 1), (dict(bt=0), 1), (dict(seq=0), 1), (dict(cdt=4), 3), (dict(cdt=1), 3),
    (dict(bdt=3, cdt=3), 3), (dict(bdt=1), 3), (dict(R=-1), 2), (dict(B=0), 2), (dict(E=0), 2), (dict(nb=-1), 2), (dict(bts=-1), 2),
    (dict(blk=-1), 2), (dict(tok=BIG), 2), (dict(bb=-1), 2), (dict(br=-1), 2), (dict(br=575), 2), (dict(bb=500), 2),
    (dict(E=1025, br=1025), 5), (dict(R=(1 << 20) + 1), 5), (dict(nb=2 ** 31), 5), (dict(bts=2 ** 31), 5), (dict(cache=4097), 4),
    (dict(bounds=4097), 4), (dict(bt=4098), 4), (dict(ctx=4098), 4), (dict(seq=4098), 4), (dict(err=4098), 4), (dict(R=0), 0),
    (dict(R=0, seq=0, cache=0), 0)])
def test_bounds_refusals(cuda_lib, over, status):
    assert cuda_lib.pmg_call_packed(4, binding.BOUNDS_ARGS.pack(*{**BOUNDS, **over}.values())) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=0), 1), (dict(bounds=0), 1), (dict(bt=0), 1), (dict(seq=0), 1), (dict(scores=0), 1), (dict(dt=3), 3), (dict(dt=9), 3),
    (dict(R=-1), 2), (dict(n=-1), 2), (dict(H=-1), 2), (dict(E=0), 2), (dict(B=0), 2), (dict(nb=-1), 2), (dict(bts=-1), 2),
    (dict(sm=-1.0), 2), (dict(sm=float("nan")), 2), (dict(opt=1), 2), (dict(qr=-1), 2), (dict(qt=BIG), 2), (dict(qh=-1), 2),
    (dict(bb=-1), 2), (dict(br=BIG), 2), (dict(ss=-1), 2), (dict(ss=3), 2), (dict(E=1025), 5), (dict(n=1 << 11, H=1 << 10), 5),
    (dict(R=(1 << 20) + 1), 5), (dict(R=1 << 20, n=1 << 11, H=0), 5), (dict(nb=2 ** 31), 5), (dict(bts=2 ** 31, ss=2 ** 31), 5),
    (dict(q=4097), 4), (dict(bounds=4097), 4), (dict(bt=4098), 4), (dict(seq=4098), 4), (dict(scale=4098), 4), (dict(lse=4098), 4),
    (dict(scores=4098), 4), (dict(err=4098), 4), (dict(R=0), 0), (dict(n=0, q=0), 0), (dict(bts=0, ss=0, bt=0), 0)])
def test_scores_refusals(cuda_lib, over, status):
    assert cuda_lib.pmg_call_packed(5, binding.SCORES_ARGS.pack(*{**SCORES, **over}.values())) == status


@pytest.mark.parametrize("over,status", [
    (dict(scores=0), 1), (dict(bt=0), 1), (dict(seq=0), 1), (dict(sel=0), 1), (dict(lens=0), 1), (dict(R=-1), 2), (dict(n=-1), 2),
    (dict(B=0), 2), (dict(bts=-1), 2), (dict(first=-1), 2), (dict(last=0), 2), (dict(first=2, last=2), 2), (dict(keep=1), 2),
    (dict(sels=2), 2), (dict(ss=3), 2), (dict(ss=BIG), 2), (dict(sels=BIG), 2), (dict(R=(1 << 20) + 1), 5),
    (dict(R=1 << 20, n=1 << 11), 5), (dict(bts=2 ** 31, ss=2 ** 31), 5), (dict(keep=2 ** 31, sels=2 ** 31), 5), (dict(scores=4098), 4),
    (dict(bt=4098), 4), (dict(seq=4098), 4), (dict(sel=4098), 4), (dict(cols=4098), 4), (dict(lens=4098), 4), (dict(err=4098), 4),
    (dict(R=0), 0), (dict(n=0, scores=0), 0)])
def test_select_refusals(cuda_lib, over, status):
    assert cuda_lib.pmg_call_packed(6, binding.SELECT_ARGS.pack(*{**SELECT, **over}.values())) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=0), 1), (dict(cache=0), 1), (dict(pt=0), 1), (dict(pl=0), 1), (dict(cu=0), 1), (dict(bt=0), 1), (dict(lens=0), 1),
    (dict(out=0), 1), (dict(ws=0), 1), (dict(qdt=3), 3), (dict(cdt=1), 3), (dict(G=-1), 2), (dict(pts=-1), 2), (dict(bts=-1), 2),
    (dict(R=-1), 2), (dict(n=-1), 2), (dict(H=-1), 2), (dict(dv=0), 2), (dict(dr=-1), 2), (dict(B=0), 2), (dict(nb=-1), 2),
    (dict(sm=-1.0), 2), (dict(opt=8), 2), *[({k: -1}, 2) for k in ("qr", "qt", "qh", "bs", "ts", "orr", "ot", "oh")],
    (dict(G=(1 << 20) + 1), 5), (dict(pts=2 ** 31), 5), (dict(dr=1000), 5), (dict(R=1 << 20, n=1 << 6, H=1 << 6), 5), (dict(q=4097), 4),
    (dict(cache=4097), 4), (dict(pt=4098), 4), (dict(pl=4098), 4), (dict(cu=4098), 4), (dict(bt=4098), 4), (dict(lens=4098), 4),
    (dict(scale=4098), 4), (dict(out=4097), 4), (dict(lse=4098), 4), (dict(ws=4104), 4), (dict(ws=4096 + 128), 4), (dict(err=4098), 4),
    (dict(R=0), 0), (dict(n=0, q=0), 0), (dict(H=0), 0)])
def test_shared_refusals(cuda_lib, over, status):
    assert cuda_lib.pmg_call_packed(7, binding.SHARED_ARGS.pack(*{**SHARED, **over}.values())) == status


def test_workspace_sizes(cuda_lib):
    assert cuda_lib.pmg_shared_workspace(-1, 512) < 0 and cuda_lib.pmg_shared_workspace(2 ** 31, 512) < 0
    assert cuda_lib.pmg_shared_workspace(1, 0) < 0 and cuda_lib.pmg_shared_workspace(1, 1025) < 0


def test_binding_refusals(cuda_lib):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i, f = torch.int32, torch.float32
    table, lens = z(2, 4, dt=i), z(2, dt=i)
    bounds = lambda **o: binding.block_bounds(**{**dict(cache=z(4, 64, 576), bounds=z(4, 2, 576), block_table=table,  # noqa: E731
                                                        seq_lens=lens), **o})
    for bad in (dict(bounds=z(4, 2, 512)), dict(bounds=z(3, 2, 576)), dict(bounds=z(4, 576, 2).transpose(1, 2)), dict(block_table=z(3, 4, dt=i)),
                dict(seq_lens=z(2)), dict(ctx_lens=z(3, dt=i)), dict(cache=z(4, 64, 576, dt=torch.float64)), dict(error_flag=z(2, dt=i))):
        with pytest.raises(ValueError):
            bounds(**bad)
    scores = lambda **o: binding.block_scores(**{**dict(q=z(2, 1, 3, 576), bounds=z(4, 2, 576), block_table=table, seq_lens=lens,  # noqa: E731
                                                        scores=z(2, 1, 4, dt=f), block_size=64, sm_scale=1.0), **o})
    for bad in (dict(q=z(2, 1, 3, 512)), dict(bounds=z(4, 3, 576)), dict(bounds=z(4, 2, 576, dt=torch.float16)), dict(scores=z(2, 1, 5, dt=f)),
                dict(scores=z(2, 1, 4)), dict(lse=z(2, 1, 2, dt=f)), dict(seq_lens=z(3, dt=i)),
                dict(q=z(2, 2, 3, 576), scores=z(2, 3, 4, dt=f)[:, :2])):
        with pytest.raises(ValueError):
            scores(**bad)
    select = lambda **o: binding.select_blocks(**{**dict(scores=z(2, 1, 4, dt=f), block_table=table, seq_lens=lens,  # noqa: E731
                                                         selected=z(2, 3, dt=i), selected_lens=z(2, dt=i), block_size=64), **o})
    for bad in (dict(selected=z(3, 3, dt=i)), dict(selected=z(2, 3)), dict(selected_lens=z(3, dt=i)), dict(scores=z(2, 1, 3, dt=f)),
                dict(columns=z(2, 4, dt=i)), dict(columns=z(2, 4, dt=i)[:, :3]), dict(scores=z(2, 1, 4))):
        with pytest.raises(ValueError):
            select(**bad)
    shared = lambda **o: binding.latent_decode_shared(**{**dict(  # noqa: E731
        q=z(2, 1, 3, 576), cache=z(4, 64, 576), prefix_table=z(1, 4, dt=i), prefix_lens=z(1, dt=i), cu_groups=z(2, dt=i), block_table=table,
        seq_lens=lens, out=z(2, 1, 3, 512), sm_scale=1.0, workspace=z(64, dt=torch.uint8)), **o})
    for bad in (dict(prefix_table=z(2, 4, dt=i)), dict(cu_groups=z(3, dt=i)), dict(prefix_lens=z(1)), dict(out=z(2, 1, 3, 600)),
                dict(out=z(2, 1, 3, 512, dt=f)), dict(cache=z(4, 64, 512)), dict(lse=z(2, 1, 2, dt=f)), dict(workspace=z(64, 2)[:, 0])):
        with pytest.raises(ValueError):
            shared(**bad)


# --- where the tensors live -----------------------------------------------------------

def bounds_args(d):
    i = lambda *s: placed(d, *s, dtype=I32)  # noqa: E731
    return binding.block_bounds, dict(cache=placed(d, 4, 64, 576), bounds=placed(d, 4, 2, 576), block_table=i(2, 4), seq_lens=i(2),
                                      ctx_lens=i(2), error_flag=i(1))


def scores_args(d):
    i = lambda *s: placed(d, *s, dtype=I32)  # noqa: E731
    return binding.block_scores, dict(q=placed(d, 2, 1, 3, 576), bounds=placed(d, 4, 2, 576), block_table=i(2, 4), seq_lens=i(2),
                                      scores=placed(d, 2, 1, 4, dtype=F32), block_size=64, sm_scale=0.1, scale=placed(d, 1, dtype=F32),
                                      lse=placed(d, 2, 1, 3, dtype=F32), error_flag=i(1))


def select_args(d):
    i = lambda *s: placed(d, *s, dtype=I32)  # noqa: E731
    return binding.select_blocks, dict(scores=placed(d, 2, 1, 4, dtype=F32), block_table=i(2, 4), seq_lens=i(2), selected=i(2, 3),
                                       selected_lens=i(2), block_size=64, columns=i(2, 3), error_flag=i(1))


def shared_args(d):
    i = lambda *s: placed(d, *s, dtype=I32)  # noqa: E731
    return binding.latent_decode_shared, dict(
        q=placed(d, 2, 1, 3, 576), cache=placed(d, 4, 64, 576), prefix_table=i(1, 4), prefix_lens=i(1), cu_groups=i(2),
        block_table=i(2, 4), seq_lens=i(2), out=placed(d, 2, 1, 3, 512), lse=placed(d, 2, 1, 3, dtype=F32), sm_scale=0.1,
        scale=placed(d, 1, dtype=F32), workspace=placed(d, 64, dtype=torch.uint8), error_flag=i(1))


CALLS = [bounds_args, scores_args, select_args, shared_args]


@pytest.mark.parametrize("args", CALLS)
def test_every_tensor_has_to_be_on_the_device(launches, args):  # noqa: F811
    devices.test_every_tensor_has_to_be_on_the_device(launches, args)


@pytest.mark.parametrize("args", CALLS)
def test_calls_run_where_their_tensors_are(launches, args):  # noqa: F811
    for device in (0, 1, 0):
        call, a = args(device)
        call(**a)
        assert launches["seen"][-1] == (4 + CALLS.index(args), device) and launches["current"] == 0
        a = {k: x for k, x in a.items() if k not in ("ctx_lens", "error_flag", "scale", "lse", "columns")}
        call(**a)
        assert launches["seen"][-1][1] == device

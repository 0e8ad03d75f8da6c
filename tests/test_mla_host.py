"""Refusals of the operators around the gather, on the host, before any CUDA call."""
import os
import re
import subprocess

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_the_operators(cuda_lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pmg_mla.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(pmg_\w+)\s*\(", text, flags=re.M)))
    assert names == ["pmg_append", "pmg_attention_workspace", "pmg_call_packed", "pmg_latent_decode", "pmg_latent_prefill",
                     "pmg_plan_step"]
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB_PATH], capture_output=True, text=True, check=True)
    for name in names:
        assert re.search(rf"\bT {name}$", out.stdout, flags=re.M)


def plan(L, **o):
    a = dict(ctx=4096, new=4096, R=2, bt=4096, bts=4, free=4096, nf=4, nb=8, B=64, slots=4096, pos=4096, t2s=4096, T=10,
             cu=4096, lens=4096, cuseq=4096, taken=4096, err=0)
    a.update(o)
    return L.pmg_plan_step(a["ctx"] or None, a["new"] or None, a["R"], a["bt"] or None, a["bts"], a["free"] or None,
                           a["nf"], a["nb"], a["B"], a["slots"] or None, a["pos"] or None, a["t2s"] or None, a["T"],
                           a["cu"] or None, a["lens"] or None, a["cuseq"] or None, a["taken"] or None, a["err"] or None,
                           None)


@pytest.mark.parametrize("over,status", [
    (dict(R=-1), 2), (dict(B=0), 2), (dict(T=-1), 2), (dict(nf=-1), 2), (dict(R=(1 << 20) + 1), 5),
    (dict(T=2 ** 31), 5), (dict(cu=0), 1), (dict(ctx=0), 1), (dict(free=0), 1), (dict(bt=0), 1), (dict(lens=0), 1),
    (dict(slots=4100), 4), (dict(ctx=4097), 4), (dict(err=2), 4)])
def test_plan_refusals(cuda_lib, over, status):
    assert plan(cuda_lib, **over) == status


def append(L, **o):
    a = dict(c=4096, cs=512, k=4096, ks=64, w=4096, eps=1e-6, rot=4096, P=10, slots=4096, pos=4096, T=4, dv=512, dr=64,
             sdt=0, cache=4096, bs=64 * 576, ts=576, nb=4, B=64, cdt=0, scale=0, q=4096, qt=64, qh=64, o=8192, ot=64,
             oh=64, H=1, err=0, opt=0)
    a.update(o)
    n = lambda k: a[k] or None  # noqa: E731
    return L.pmg_append(n("c"), a["cs"], n("k"), a["ks"], n("w"), a["eps"], n("rot"), a["P"], n("slots"), n("pos"),
                        a["T"], a["dv"], a["dr"], a["sdt"], n("cache"), a["bs"], a["ts"], a["nb"], a["B"], a["cdt"],
                        n("scale"), n("q"), a["qt"], a["qh"], n("o"), a["ot"], a["oh"], a["H"], n("err"), None, a["opt"])


@pytest.mark.parametrize("over,status", [
    (dict(sdt=3), 3), (dict(sdt=9), 3), (dict(cdt=4), 3), (dict(dr=3), 2), (dict(dv=0), 2), (dict(B=0), 2),
    (dict(cs=-1), 2), (dict(opt=2), 2), (dict(eps=float("nan")), 2), (dict(eps=-1.0), 2), (dict(H=-1), 2),
    (dict(T=2 ** 31), 5), (dict(c=0), 1), (dict(slots=0), 1), (dict(pos=0), 1), (dict(cache=0), 1), (dict(rot=0), 1),
    (dict(q=0), 1), (dict(o=0), 1), (dict(k=0), 1), (dict(c=4097), 4), (dict(slots=4100), 4), (dict(w=4098), 4),
    (dict(T=0), 0), (dict(T=0, c=0, slots=0), 0)])
def test_append_refusals(cuda_lib, over, status):
    assert append(cuda_lib, **over) == status


def decode(L, **o):
    a = dict(q=4096, qr=576, qt=576, qh=576, cache=4096, bs=64 * 576, ts=576, nb=4, bt=4096, bts=4, lens=4096, R=2, n=1,
             H=1, dv=512, dr=64, B=64, qdt=0, cdt=0, scale=0, sm=0.1, out=4096, orr=512, ot=512, oh=512, lse=4096,
             ws=4096, wsb=1 << 40, err=0, opt=0)
    a.update(o)
    n = lambda k: a[k] or None  # noqa: E731
    return L.pmg_latent_decode(n("q"), a["qr"], a["qt"], a["qh"], n("cache"), a["bs"], a["ts"], a["nb"], n("bt"),
                               a["bts"], n("lens"), a["R"], a["n"], a["H"], a["dv"], a["dr"], a["B"], a["qdt"],
                               a["cdt"], n("scale"), a["sm"], n("out"), a["orr"], a["ot"], a["oh"], n("lse"), n("ws"),
                               a["wsb"], n("err"), None, a["opt"])


@pytest.mark.parametrize("over,status", [
    (dict(qdt=3), 3), (dict(cdt=1), 3), (dict(qdt=1, cdt=0), 3), (dict(cdt=4), 3), (dict(R=-1), 2), (dict(n=-1), 2),
    (dict(dv=0), 2), (dict(B=0), 2), (dict(sm=float("nan")), 2), (dict(sm=-1.0), 2), (dict(opt=1), 2), (dict(qr=-1), 2),
    (dict(dv=1000, dr=64), 5), (dict(n=1 << 11, H=1 << 10), 5), (dict(R=(1 << 20) + 1), 5), (dict(q=0), 1),
    (dict(cache=0), 1), (dict(bt=0), 1), (dict(lens=0), 1), (dict(out=0), 1), (dict(ws=0), 1), (dict(q=4097), 4),
    (dict(ws=4104), 4), (dict(lse=4098), 4), (dict(R=0), 0), (dict(H=0), 0), (dict(n=0, q=0), 0)])
def test_decode_refusals(cuda_lib, over, status):
    assert decode(cuda_lib, **over) == status


def prefill(L, **o):
    a = dict(q=4096, qt=192, qh=192, k=4096, kt=256, kh=256, pe=4096, ps=64, v=4096, vt=256, vh=256, cq=4096, ck=4096,
             R=1, Tq=4, Tk=4, H=1, dn=128, dr=64, dv=128, dt=0, sm=0.1, out=4096, ot=128, oh=128, lse=0, prev=0, pt=0,
             ph=0, pl=0, ws=4096, wsb=1 << 40, err=0, opt=0)
    a.update(o)
    n = lambda k: a[k] or None  # noqa: E731
    return L.pmg_latent_prefill(n("q"), a["qt"], a["qh"], n("k"), a["kt"], a["kh"], n("pe"), a["ps"], n("v"), a["vt"],
                                a["vh"], n("cq"), n("ck"), a["R"], a["Tq"], a["Tk"], a["H"], a["dn"], a["dr"], a["dv"],
                                a["dt"], a["sm"], n("out"), a["ot"], a["oh"], n("lse"), n("prev"), a["pt"], a["ph"],
                                n("pl"), n("ws"), a["wsb"], n("err"), None, a["opt"])


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), 3), (dict(dt=4), 3), (dict(R=-1), 2), (dict(dn=0), 2), (dict(dv=0), 2), (dict(qt=-1), 2),
    (dict(sm=float("nan")), 2), (dict(opt=4), 2), (dict(dn=1000), 5), (dict(dv=1025), 5), (dict(Tq=2 ** 31), 5),
    (dict(q=0), 1), (dict(k=0), 1), (dict(pe=0), 1), (dict(v=0), 1), (dict(cq=0), 1), (dict(ws=0), 1),
    (dict(prev=4096), 1), (dict(pl=4096), 1), (dict(q=4097), 4), (dict(ws=4104), 4), (dict(R=0), 0), (dict(Tq=0), 0)])
def test_prefill_refusals(cuda_lib, over, status):
    assert prefill(cuda_lib, **over) == status


def test_binding_refusals(cuda_lib):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = torch.int32
    with pytest.raises(ValueError):  # entry sizes differ
        binding.latent_decode(z(1, 1, 2, 576), z(4, 64, 512), z(1, 4, dt=i), z(1, dt=i), z(1, 1, 2, 512), sm_scale=1.0,
                              workspace=z(16))
    with pytest.raises(ValueError):  # table of another batch
        binding.latent_decode(z(1, 1, 2, 576), z(4, 64, 576), z(2, 4, dt=i), z(1, dt=i), z(1, 1, 2, 512), sm_scale=1.0,
                              workspace=z(16))
    with pytest.raises(ValueError):  # one of two
        binding.latent_prefill(z(4, 2, 192), z(4, 2, 128), z(4, 64), z(4, 2, 128), z(2, dt=i), z(2, dt=i),
                               z(4, 2, 128), sm_scale=1.0, prev_out=z(4, 2, 128), workspace=z(16))
    with pytest.raises(ValueError):  # slots of another type
        binding.append(z(4, 512), z(4, 64), z(2, 16, 576), z(4, dt=i), z(4, dt=i), z(9, 64, dt=torch.float32))
    with pytest.raises(ValueError):
        binding.plan_step(z(2, dt=i), z(3, dt=i), z(2, 4, dt=i), z(4, dt=i), 16, None, None, None, z(3, dt=i),
                          z(2, dt=i), None, None, 4)


def test_packed_calls_pass_every_argument(cuda_lib):
    """Each argument in turn, out of range, gives its own refusal through the packed call: none is lost or shifted."""
    decode = dict(binding.DECODE_WORDS)  # name -> format, in order
    good = dict(q=4096, q_req_stride=576, q_token_stride=576, q_head_stride=576, cache=4096, cache_block_stride=64 * 576,
                cache_token_stride=576, num_blocks=4, block_table=4096, block_table_stride=4, seq_lens=4096, num_reqs=2,
                q_len=1, heads=1, latent_dim=512, rope_dim=64, block_size=64, q_dtype=0, cache_dtype=0, scale=0,
                sm_scale=0.1, out=4096, out_req_stride=512, out_token_stride=512, out_head_stride=512, lse=4096,
                workspace=4096, workspace_bytes=0, error_flag=0, stream=0, options=0)
    assert list(decode) == list(good)

    def run(**over):
        return cuda_lib.pmg_call_packed(2, binding.DECODE_ARGS.pack(*{**good, **over}.values()))
    for name, value, status in [("q", 0, 1), ("q", 4097, 4), ("cache", 0, 1), ("cache", 4097, 4), ("block_table", 4098, 4),
                                ("seq_lens", 0, 1), ("num_reqs", -1, 2), ("q_len", -1, 2), ("heads", -1, 2),
                                ("latent_dim", 0, 2), ("rope_dim", -1, 2), ("rope_dim", 1000, 5), ("block_size", 0, 2),
                                ("q_dtype", 9, 3), ("cache_dtype", 9, 3), ("scale", 2, 4), ("sm_scale", -1.0, 2),
                                ("out", 0, 1), ("lse", 2, 4), ("workspace", 0, 1), ("workspace", 8, 4),
                                ("error_flag", 2, 4), ("options", 8, 2), ("num_blocks", -1, 2), ("block_table_stride", -1, 2),
                                *[(n, -1, 2) for n in good if n.endswith("_stride") and n != "block_table_stride"]]:
        assert run(**{name: value}) == status, name
    assert cuda_lib.pmg_call_packed(2, None) == 1 and cuda_lib.pmg_call_packed(9, b"12345678") == 2
    assert len(binding.PLAN_ARGS.pack(*[0] * 19)) == 19 * 8
    assert cuda_lib.pmg_call_packed(0, binding.PLAN_ARGS.pack(*[0] * 8, 0, *[0] * 10)) == 2  # block_size 0
    assert cuda_lib.pmg_call_packed(1, binding.APPEND_ARGS.pack(*[0] * 5, 0.0, *[0] * 25)) == 2
    assert cuda_lib.pmg_call_packed(3, binding.PREFILL_ARGS.pack(*[0] * 21, 0.0, *[0] * 13)) == 2

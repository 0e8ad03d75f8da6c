"""Where the tensors of the operators around the gather live: checked before their addresses go anywhere."""
import contextlib

import pytest
import torch

from paged_mla_kv_cache_gb300 import binding

BF16, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


class Placed(torch.Tensor):
    """A host tensor that says it is on cuda:`where` (None: pinned host memory, -1: ordinary host memory)."""

    @property
    def is_cuda(self):
        return self.where is not None and self.where >= 0

    def get_device(self):
        return self.where if self.is_cuda else -1

    def is_pinned(self):
        return self.where is None


def placed(where, *shape, dtype=BF16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Placed)
    t.where = where
    return t


def plan_args(d):
    i = lambda *s: placed(d, *s, dtype=I32)  # noqa: E731
    a = dict(ctx_lens=i(2), new_lens=i(2), block_table=i(2, 4), free_blocks=i(4), block_size=16,
             slots=placed(d, 5, dtype=I64), positions=i(5), token_to_seq=i(5), cu_new=i(3), seq_lens=i(2), cu_seq=i(3),
             blocks_taken=i(1), num_blocks=9, error_flag=i(1))
    return binding.plan_step, a


def append_args(d):
    a = dict(c_kv=placed(d, 4, 512), k_pe=placed(d, 4, 64), cache=placed(d, 2, 16, 576), slots=placed(d, 4, dtype=I64),
             positions=placed(d, 4, dtype=I32), cos_sin=placed(d, 9, 64, dtype=F32), norm_weight=placed(d, 512, dtype=F32),
             scale=placed(d, 1, dtype=F32), q_pe=placed(d, 4, 3, 64), q_out=placed(d, 4, 3, 64),
             error_flag=placed(d, 1, dtype=I32))
    return binding.append, a


def decode_args(d):
    a = dict(q=placed(d, 2, 1, 4, 576), cache=placed(d, 4, 64, 576), block_table=placed(d, 2, 4, dtype=I32),
             seq_lens=placed(d, 2, dtype=I32), out=placed(d, 2, 1, 4, 512), lse=placed(d, 2, 1, 4, dtype=F32), sm_scale=0.1,
             scale=placed(d, 1, dtype=F32), workspace=placed(d, 64, dtype=torch.uint8), error_flag=placed(d, 1, dtype=I32))
    return binding.latent_decode, a


def prefill_args(d):
    a = dict(q=placed(d, 4, 2, 192), k_nope=placed(d, 6, 2, 128), k_pe=placed(d, 6, 64), v=placed(d, 6, 2, 128),
             cu_q=placed(d, 2, dtype=I32), cu_k=placed(d, 2, dtype=I32), out=placed(d, 4, 2, 128),
             lse=placed(d, 4, 2, dtype=F32), sm_scale=0.1, prev_out=placed(d, 4, 2, 128), prev_lse=placed(d, 4, 2, dtype=F32),
             workspace=placed(d, 64, dtype=torch.uint8), error_flag=placed(d, 1, dtype=I32))
    return binding.latent_prefill, a


CALLS = [plan_args, append_args, decode_args, prefill_args]


@pytest.fixture
def launches(monkeypatch):
    """Two devices, cuda:0 current, and a library that notes the device that is current at each call."""
    state = dict(current=0, seen=[], devices=2)

    class Library:
        @staticmethod
        def pmg_call_packed(which, words):
            state["seen"].append((which, state["current"]))
            return 0

    @contextlib.contextmanager
    def on(device):
        before, state["current"] = state["current"], int(device)
        yield
        state["current"] = before

    monkeypatch.setattr(binding, "load_library", lambda: Library)
    monkeypatch.setattr(binding, "_one_device", False, raising=False)
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: state["devices"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", on)
    return state


@pytest.mark.parametrize("args", CALLS)
def test_every_tensor_has_to_be_on_the_device(launches, args):
    tensors = [k for k, x in args(0)[1].items() if isinstance(x, torch.Tensor)]
    for devices in (1, 2):
        launches["devices"], binding._one_device = devices, False
        for name in tensors:
            call, a = args(0)
            call(**a)  # as it should be
            for where in (-1, 1) if devices == 2 else (-1,):
                b = dict(a)
                b[name] = a[name].clone().as_subclass(Placed)
                b[name].where = where
                before = len(launches["seen"])
                with pytest.raises(ValueError):
                    call(**b)
                assert len(launches["seen"]) == before
    call, a = args(-1)
    with pytest.raises(ValueError):
        call(**a)


@pytest.mark.parametrize("args", CALLS)
def test_calls_run_where_their_tensors_are(launches, args):
    which = CALLS.index(args)
    for device in (0, 1, 0):
        call, a = args(device)
        call(**a)
        assert launches["seen"][-1] == (which, device) and launches["current"] == 0


def test_pinned_host_memory_is_taken(launches):
    """Every device reaches it: a host that polls the flag or the count keeps them there."""
    for args in CALLS:
        call, a = args(1)
        a["error_flag"].where = None
        if "blocks_taken" in a:
            a["blocks_taken"].where = None
        call(**a)
        assert launches["seen"][-1][1] == 1


def test_optional_tensors_may_be_absent(launches):
    for args, names in ((plan_args, ("slots", "positions", "token_to_seq", "cu_seq", "blocks_taken", "error_flag")),
                        (append_args, ("norm_weight", "scale", "q_pe", "q_out", "error_flag")),
                        (decode_args, ("lse", "scale", "error_flag")),
                        (prefill_args, ("lse", "prev_out", "prev_lse", "error_flag"))):
        for device in (0, 1):
            call, a = args(device)
            call(**{**a, **{n: None for n in names}})
            assert launches["seen"][-1][1] == device


@pytest.mark.parametrize("args", [decode_args, prefill_args])
def test_workspace_is_one_piece(launches, args):
    call, a = args(0)
    a["workspace"] = placed(0, 64, 2, dtype=torch.uint8)[:, 0]
    a["workspace"].where = 0
    with pytest.raises(ValueError):
        call(**a)

"""Thin ctypes binding of ``libpmg.so`` (declared in ``include/pmg.h``,
``include/pmg_mla.h`` and ``include/pmg_long.h``).

Argument marshalling only: shapes, strides, dtypes and raw pointers are taken
from torch tensors and passed to the C ABI; every step of the gather runs in
the CUDA kernels of ``csrc/pmg_gather.cu``. There is no fallback: if the
library is missing or a call fails, a PmgError is raised.

The call mirrors ops.cp_gather_cache(src_cache, dst, block_table, cu_seq_lens,
batch_size, seq_starts) of "MLA cache gather scheduled per logical page"
(prhub.com.cn, vllm PR #51739, section "关键源码片段"), with the dtype pair,
the FP8 scale, an error flag and the stream made explicit.

plan_step, append, latent_decode and latent_prefill are the operators around
the gather: a step's pages and slots, the cache write, and the attention over
the cache (absorbed) or over gathered and expanded entries. block_bounds,
block_scores and select_blocks choose the pages of a long request that a token
attends to, and latent_decode_shared attends behind prefixes that requests share.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Tuple

import torch

from .build import LIB_PATH

PMG_OK = 0
STATUS_NAMES = {0: "PMG_OK", 1: "PMG_ERR_NULL", 2: "PMG_ERR_ARG", 3: "PMG_ERR_DTYPE", 4: "PMG_ERR_ALIGN",
                5: "PMG_ERR_UNSUPPORTED", 6: "PMG_ERR_CUDA"}

DTYPE_CODES = {"bf16": 0, "fp16": 1, "fp32": 2, "fp8_e4m3": 3, "u8": 4}
TORCH_DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3, torch.uint8: 4}

FLAG_LOGICAL_BLOCK = 1
FLAG_PHYS_BLOCK = 2
FLAG_SEQ_START = 4
FLAG_CU_ORDER = 8
FLAG_TIMEOUT = 16
FLAG_TOKEN = 32
FLAG_LENGTH = 64
FLAG_CAPACITY = 128
FLAG_NO_BLOCKS = 256
FLAG_POSITION = 512

OPT_FORCE_SIMT = 1
OPT_FORCE_SCALAR = 2
OPT_IMPLIED_END = 4
OPT_EARLY_METADATA = 8
OPT_ROPE_PAIRS = 1         # append
OPT_CAUSAL = 1             # latent_prefill
OPT_FORCE_GENERAL = 2      # latent_decode, latent_prefill, block_scores, latent_decode_shared
MAX_ENTRY = 1024           # largest latent_dim + rope_dim of the attention calls

PATH_NAMES = {0: "none", 1: "bulk", 2: "vector", 3: "scalar", 4: "realign"}
WORKSPACE_INTS = 4
MAX_REQS_PLAN = 4096       # requests one launch plans; more need a workspace
MAX_REQS = 1 << 20         # requests one call accepts


class PmgError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status})")


_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libpmg.so once. Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise PmgError(6, f"CUDA library {LIB_PATH} is missing; build it with "
                              "paged_mla_kv_cache_gb300.build.build_library()")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, u32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_void_p
        gather_args = [vp, i64, i64, i64, vp, i64, vp, vp, i32, i64, i32, i32, i32, i32, vp, vp, i64, vp, vp]
        L.pmg_gather.restype = ctypes.c_int
        L.pmg_gather.argtypes = gather_args
        L.pmg_gather_ex.restype = ctypes.c_int
        L.pmg_gather_ex.argtypes = gather_args[:18] + [vp, vp, u32]
        L.pmg_gather_noalloc.restype = ctypes.c_int
        L.pmg_gather_noalloc.argtypes = gather_args
        L.pmg_debug_noalloc_scratch.restype = ctypes.c_int
        L.pmg_debug_noalloc_scratch.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(i64)]
        L.pmg_gather_tokens.restype = ctypes.c_int
        L.pmg_gather_tokens.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp, i32, i64, i32, i32, i32, i32, vp, vp, i64,
                                        vp, vp, vp, u32]
        L.pmg_select_path.restype = ctypes.c_int
        L.pmg_select_path.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, i64, i32, i32, i32, i32, vp, i64, u32,
                                      ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.pmg_debug_plan.restype = ctypes.c_int
        L.pmg_debug_plan.argtypes = [vp, vp, i32, i64, i32, vp, i64, vp, vp, vp, u32]
        f32 = ctypes.c_float
        L.pmg_plan_step.restype = ctypes.c_int
        L.pmg_plan_step.argtypes = [vp, vp, i32, vp, i64, vp, i64, i64, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp]
        L.pmg_append.restype = ctypes.c_int
        L.pmg_append.argtypes = [vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, i64, i32, i32, i32, vp, i64, i64, i64, i32,
                                 i32, vp, vp, i64, i64, vp, i64, i64, i32, vp, vp, u32]
        L.pmg_latent_decode.restype = ctypes.c_int
        L.pmg_latent_decode.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64, vp, i64, vp, i32, i32, i32, i32, i32, i32,
                                        i32, i32, vp, f32, vp, i64, i64, i64, vp, vp, i64, vp, vp, u32]
        L.pmg_latent_prefill.restype = ctypes.c_int
        L.pmg_latent_prefill.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, i32, i64, i64, i32,
                                         i32, i32, i32, i32, f32, vp, i64, i64, vp, vp, i64, i64, vp, vp, i64, vp, vp,
                                         u32]
        L.pmg_block_bounds.restype = ctypes.c_int
        L.pmg_block_bounds.argtypes = [vp, i64, i64, i64, i32, i32, i32, vp, i64, i64, i32, vp, i64, vp, vp, i32, vp, vp]
        L.pmg_block_scores.restype = ctypes.c_int
        L.pmg_block_scores.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64, vp, i64, vp, i32, i32, i32, i32, i32, i32,
                                       vp, f32, vp, vp, i64, vp, vp, u32]
        L.pmg_select_blocks.restype = ctypes.c_int
        L.pmg_select_blocks.argtypes = [vp, i64, vp, i64, vp, i32, i32, i32, vp, i64, vp, vp, i64, i32, i32, vp, vp]
        L.pmg_latent_decode_shared.restype = ctypes.c_int
        L.pmg_latent_decode_shared.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64, vp, i64, vp, vp, i32, vp, i64, vp,
                                               i32, i32, i32, i32, i32, i32, i32, i32, vp, f32, vp, i64, i64, i64, vp,
                                               vp, i64, vp, vp, u32]
        L.pmg_shared_workspace.restype = i64
        L.pmg_shared_workspace.argtypes = [i64, i32]
        L.pmg_call_packed.restype = ctypes.c_int
        L.pmg_call_packed.argtypes = [i32, ctypes.c_char_p]
        L.pmg_attention_workspace.restype = i64
        L.pmg_attention_workspace.argtypes = []
        L.pmg_status_string.restype = ctypes.c_char_p
        L.pmg_status_string.argtypes = [ctypes.c_int]
        L.pmg_version.restype = ctypes.c_int
        L.pmg_version.argtypes = []
        _lib = L
        return _lib


def status_string(status: int) -> str:
    return load_library().pmg_status_string(status).decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _table_width(block_table: torch.Tensor) -> int:
    if block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise ValueError("block_table must be int32 [num_reqs, block_table_stride]")
    if block_table.shape[0] > 1 and block_table.stride(0) != block_table.shape[1] or (
            block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be contiguous")
    return block_table.shape[1]


def _layout(cache: torch.Tensor, dst: torch.Tensor):
    if cache.dim() != 3:
        raise ValueError("cache must be [num_blocks, block_size, entry_size] (a padded row is a strided view)")
    if dst.dim() != 2:
        raise ValueError("dst must be [total_tokens, entry_size]")
    if cache.shape[2] > 1 and cache.stride(2) != 1 or dst.shape[1] > 1 and dst.stride(1) != 1:
        raise ValueError("the entry dimension must be contiguous")
    if cache.dtype not in TORCH_DTYPE_CODES or dst.dtype not in TORCH_DTYPE_CODES:
        raise ValueError(f"unsupported dtype {cache.dtype} -> {dst.dtype}")
    return TORCH_DTYPE_CODES[cache.dtype], TORCH_DTYPE_CODES[dst.dtype]


def gather(cache: torch.Tensor, dst: torch.Tensor, block_table: torch.Tensor, cu_seq_lens: torch.Tensor,
           seq_starts: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
           error_flag: Optional[torch.Tensor] = None, num_reqs: Optional[int] = None, stream=None,
           options: int = 0, workspace: Optional[torch.Tensor] = None) -> None:
    """Gather the cached entries of every request into dst (asynchronous).

    cache        [num_blocks, block_size, entry_size] device tensor; a padded
                 row stride is expressed as a view (stride(1) > entry_size).
    dst          [total_tokens, entry_size] device tensor (may be a row-strided view).
    block_table  int32 [num_reqs, block_table_stride]; row stride = stride(0).
    cu_seq_lens  int32 [num_reqs + 1] (or [num_reqs] with OPT_IMPLIED_END).
    seq_starts   int32 [num_reqs] or None.
    scale        fp32 device scalar tensor or None (1.0); used for fp8 sources.
    error_flag   int32 device tensor of one element or None.
    num_reqs     defaults to the request count implied by cu_seq_lens.
    workspace    int32 device tensor of WORKSPACE_INTS zeros (see new_workspace), or
                 None: dynamic work distribution on the TMA paths.
    """
    src_code, dst_code = _layout(cache, dst)
    if num_reqs is None:
        num_reqs = cu_seq_lens.shape[0] - (0 if options & OPT_IMPLIED_END else 1)
    bt_stride = _table_width(block_table)
    st = load_library().pmg_gather_ex(
        _ptr(cache), cache.stride(0), cache.stride(1), cache.shape[0],
        _ptr(block_table), bt_stride, _ptr(cu_seq_lens), _ptr(seq_starts), int(num_reqs),
        dst.shape[0], cache.shape[1], cache.shape[2], src_code, dst_code, _ptr(scale),
        _ptr(dst), dst.stride(0), _ptr(error_flag), _ptr(workspace),
        _stream_handle(stream), int(options))
    if st != PMG_OK:
        raise PmgError(st, "pmg_gather")


def gather_noalloc(cache: torch.Tensor, dst: torch.Tensor, block_table: torch.Tensor, cu_seq_lens: torch.Tensor,
                   seq_starts: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                   error_flag: Optional[torch.Tensor] = None, num_reqs: Optional[int] = None, stream=None) -> None:
    """gather() for callers that cannot allocate device memory: the dynamic
    work split runs on the library's own static scratch instead of a caller
    workspace (pmg_gather_noalloc). Calls that overlap on the GPU must not use
    it concurrently; make the first call on a device outside stream capture."""
    src_code, dst_code = _layout(cache, dst)
    if num_reqs is None:
        num_reqs = cu_seq_lens.shape[0] - 1
    st = load_library().pmg_gather_noalloc(
        _ptr(cache), cache.stride(0), cache.stride(1), cache.shape[0],
        _ptr(block_table), _table_width(block_table), _ptr(cu_seq_lens), _ptr(seq_starts), int(num_reqs),
        dst.shape[0], cache.shape[1], cache.shape[2], src_code, dst_code, _ptr(scale),
        _ptr(dst), dst.stride(0), _ptr(error_flag), _stream_handle(stream))
    if st != PMG_OK:
        raise PmgError(st, "pmg_gather_noalloc")


def debug_noalloc_scratch() -> Tuple[int, int]:
    """(device address, int32 elements) of the static scratch that
    gather_noalloc uses on the current device (pmg_debug_noalloc_scratch); a
    test hook."""
    ptr = ctypes.c_void_p()
    n = ctypes.c_int64()
    st = load_library().pmg_debug_noalloc_scratch(ctypes.byref(ptr), ctypes.byref(n))
    if st != PMG_OK:
        raise PmgError(st, "pmg_debug_noalloc_scratch")
    return int(ptr.value), int(n.value)


def gather_tokens(cache: torch.Tensor, dst: torch.Tensor, block_table: torch.Tensor, token_to_seq: torch.Tensor,
                  cu_seq_lens: torch.Tensor, scale: Optional[torch.Tensor] = None,
                  error_flag: Optional[torch.Tensor] = None, num_reqs: Optional[int] = None, stream=None,
                  options: int = 0, workspace: Optional[torch.Tensor] = None) -> None:
    """Per-token indexed gather (pmg_gather_tokens): dst row t comes from
    request token_to_seq[t] at position t - cu_seq_lens[token_to_seq[t]].
    dst has num_tokens = len(token_to_seq) rows used. workspace as in gather()."""
    src_code, dst_code = _layout(cache, dst)
    if num_reqs is None:
        num_reqs = cu_seq_lens.shape[0] - 1
    st = load_library().pmg_gather_tokens(
        _ptr(cache), cache.stride(0), cache.stride(1), cache.shape[0],
        _ptr(block_table), _table_width(block_table), _ptr(token_to_seq), _ptr(cu_seq_lens), int(num_reqs),
        token_to_seq.shape[0], cache.shape[1], cache.shape[2], src_code, dst_code, _ptr(scale),
        _ptr(dst), dst.stride(0), _ptr(error_flag), _ptr(workspace), _stream_handle(stream), int(options))
    if st != PMG_OK:
        raise PmgError(st, "pmg_gather_tokens")


def new_workspace(device) -> torch.Tensor:
    """A zeroed scheduling workspace for gather(..., workspace=...). One per
    stream: concurrent calls must not share one."""
    return torch.zeros(WORKSPACE_INTS, dtype=torch.int32, device=device)


def select_path(cache: torch.Tensor, dst: torch.Tensor, block_table: torch.Tensor, cu_seq_lens: torch.Tensor,
                num_reqs: Optional[int] = None, options: int = 0) -> Tuple[str, int]:
    """The path and access width (elements) pmg_gather_ex would use. Host only:
    tensors may live anywhere, only their pointers' alignment is looked at."""
    src_code, dst_code = _layout(cache, dst)
    if num_reqs is None:
        num_reqs = cu_seq_lens.shape[0] - (0 if options & OPT_IMPLIED_END else 1)
    path = ctypes.c_int32(-1)
    unit = ctypes.c_int32(-1)
    bt_stride = _table_width(block_table)
    st = load_library().pmg_select_path(
        _ptr(cache), cache.stride(0), cache.stride(1), cache.shape[0], _ptr(block_table), bt_stride,
        _ptr(cu_seq_lens), int(num_reqs), dst.shape[0], cache.shape[1], cache.shape[2], src_code, dst_code,
        _ptr(dst), dst.stride(0), int(options),
        ctypes.byref(path), ctypes.byref(unit))
    if st != PMG_OK:
        raise PmgError(st, "pmg_select_path")
    return PATH_NAMES[path.value], unit.value


def debug_plan(cu_seq_lens: torch.Tensor, seq_starts: Optional[torch.Tensor], total_tokens: int, block_size: int,
               max_tasks: int, error_flag: Optional[torch.Tensor] = None, num_reqs: Optional[int] = None,
               stream=None, options: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Run the device page-task mapper alone. Returns (tasks int32 [max_tasks, 5],
    num_tasks int64 [1]) as device tensors; rows past num_tasks are untouched (-1)."""
    dev = cu_seq_lens.device
    if num_reqs is None:
        num_reqs = cu_seq_lens.shape[0] - (0 if options & OPT_IMPLIED_END else 1)
    tasks = torch.full((max(max_tasks, 0), 5), -1, dtype=torch.int32, device=dev)
    num = torch.full((1,), -1, dtype=torch.int64, device=dev)
    st = load_library().pmg_debug_plan(
        _ptr(cu_seq_lens), _ptr(seq_starts), int(num_reqs), int(total_tokens), int(block_size),
        _ptr(tasks) if max_tasks > 0 else None, int(max_tasks), _ptr(num), _ptr(error_flag),
        _stream_handle(stream), int(options))
    if st != PMG_OK:
        raise PmgError(st, "pmg_debug_plan")
    return tasks, num


# --- the operators around the gather (include/pmg_mla.h) -------------------------


# Their arguments travel as one array of words (pmg_call_packed): passing thirty
# of them one by one costs ctypes more than a short call takes on the GPU. For
# the same reason the checks below first test everything in one expression and
# look for what is wrong only then.
PLAN_ARGS = struct.Struct("<19q")
APPEND_ARGS = struct.Struct("<5qd25q")
DECODE_WORDS = [(n, "d" if n == "sm_scale" else "q") for n in (
    "q q_req_stride q_token_stride q_head_stride cache cache_block_stride cache_token_stride num_blocks block_table "
    "block_table_stride seq_lens num_reqs q_len heads latent_dim rope_dim block_size q_dtype cache_dtype scale sm_scale "
    "out out_req_stride out_token_stride out_head_stride lse workspace workspace_bytes error_flag stream options").split()]
DECODE_ARGS = struct.Struct("<" + "".join(f for _, f in DECODE_WORDS))
PREFILL_ARGS = struct.Struct("<21qd13q")
BOUNDS_ARGS = struct.Struct("<18q")
SCORES_ARGS = struct.Struct("<18qd6q")
SELECT_ARGS = struct.Struct("<17q")
SHARED_ARGS = struct.Struct("<25qd10q")
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


_one_device = False  # known that this process sees one device: what is on a device is on that one


def _same_device(**tensors: Optional[torch.Tensor]) -> int:
    """The device of a call's tensors: one for all of them, or pinned host memory, which every device reaches."""
    global _one_device
    device = None
    for what, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            if not t.is_pinned():
                raise ValueError(f"{what} must be on a CUDA device, got {t.device}")
        elif device is None:
            device = t.get_device()
        elif t.get_device() != device:
            raise ValueError(f"{what} is on {t.device}, other tensors are on cuda:{device}")
    if device is None:
        raise ValueError("no tensor is on a CUDA device")
    _one_device = torch.cuda.device_count() == 1
    return device


def _call(which: int, words: bytes, device: int) -> int:
    """pmg_call_packed with `device` current: the library launches there."""
    if torch.cuda.current_device() == device:
        return load_library().pmg_call_packed(which, words)
    with torch.cuda.device(device):
        return load_library().pmg_call_packed(which, words)


def _is_vector(t: torch.Tensor, dtype: torch.dtype, n: int) -> bool:
    return t.dtype is dtype and t.numel() == n and t.is_contiguous()


def _vector(t: Optional[torch.Tensor], dtype: torch.dtype, n: int, what: str, optional: bool = False) -> None:
    if t is None:
        if not optional:
            raise ValueError(f"{what} is required")
    elif not _is_vector(t, dtype, n):
        raise ValueError(f"{what} must be {n} contiguous {dtype}, got {t.dtype} {list(t.shape)}")


def _scalar(t: Optional[torch.Tensor], dtype: torch.dtype, what: str) -> int:
    if t is None:
        return 0
    if t.dtype is not dtype or t.numel() != 1:
        raise ValueError(f"{what} must be one {dtype} element")
    return t.data_ptr()


def _unit_last(what: str, dims: int, t: torch.Tensor):
    """Shape and strides of a tensor whose last dimension is contiguous."""
    shape, strides = t.shape, t.stride()
    if len(shape) != dims or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{what} must have {dims} dimensions, the last of stride 1")
    return shape, strides


def _table(block_table: torch.Tensor, reqs: int) -> int:
    if block_table.dtype is _I32 and block_table.is_contiguous():
        shape = block_table.shape
        if len(shape) == 2 and shape[0] == reqs:
            return shape[1]
    width = _table_width(block_table)
    if block_table.shape[0] != reqs:
        raise ValueError(f"block_table has {block_table.shape[0]} rows for {reqs} requests")
    return width


def plan_step(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_blocks: torch.Tensor,
              block_size: int, slots: Optional[torch.Tensor], positions: Optional[torch.Tensor],
              token_to_seq: Optional[torch.Tensor], cu_new: torch.Tensor, seq_lens: torch.Tensor,
              cu_seq: Optional[torch.Tensor], blocks_taken: Optional[torch.Tensor], num_blocks: int,
              error_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Block table, slots and positions of one serving step (pmg_plan_step).

    ctx_lens, new_lens  int32 [num_reqs]: tokens in the cache, tokens joining.
    block_table   int32 [num_reqs, width]: the columns of fresh pages are
                  filled with ids from free_blocks (int32 [num_free]), in the
                  order of requests and pages.
    slots         int64 [max_tokens] or None: block id * block_size + offset
                  of each new token; -1 without a page and past the last token.
    positions, token_to_seq  int32 [max_tokens] or None (-1 past the last token).
    cu_new, cu_seq  int32 [num_reqs + 1]: prefix sums of new and total lengths
                  (cu_seq is the gather's cu_seq_lens; it may be None).
    seq_lens      int32 [num_reqs]: total lengths, in memory of their own: no
                  result may overlap ctx_lens, new_lens or free_blocks.
    blocks_taken  int32 [1] or None.
    """
    r = ctx_lens.numel()
    first = slots if slots is not None else positions if positions is not None else token_to_seq
    tokens = 0 if first is None else first.numel()
    free = free_blocks.numel()
    if not (_is_vector(ctx_lens, _I32, r) and _is_vector(new_lens, _I32, r) and _is_vector(free_blocks, _I32, free)
            and _is_vector(cu_new, _I32, r + 1) and _is_vector(seq_lens, _I32, r)
            and (slots is None or _is_vector(slots, _I64, tokens))
            and (positions is None or _is_vector(positions, _I32, tokens))
            and (token_to_seq is None or _is_vector(token_to_seq, _I32, tokens))
            and (cu_seq is None or _is_vector(cu_seq, _I32, r + 1))):
        for what, t, dtype, n, optional in (
                ("ctx_lens", ctx_lens, _I32, r, False), ("new_lens", new_lens, _I32, r, False),
                ("free_blocks", free_blocks, _I32, free, False), ("cu_new", cu_new, _I32, r + 1, False),
                ("seq_lens", seq_lens, _I32, r, False), ("slots", slots, _I64, tokens, True),
                ("positions", positions, _I32, tokens, True), ("token_to_seq", token_to_seq, _I32, tokens, True),
                ("cu_seq", cu_seq, _I32, r + 1, True)):
            _vector(t, dtype, n, what, optional)
    width, taken = _table(block_table, r), _scalar(blocks_taken, _I32, "blocks_taken")
    flag = _scalar(error_flag, _I32, "error_flag")
    device = 0
    if not (_one_device and ctx_lens.is_cuda and new_lens.is_cuda and block_table.is_cuda and free_blocks.is_cuda
            and cu_new.is_cuda and seq_lens.is_cuda and (slots is None or slots.is_cuda)
            and (positions is None or positions.is_cuda) and (token_to_seq is None or token_to_seq.is_cuda)
            and (cu_seq is None or cu_seq.is_cuda) and (blocks_taken is None or blocks_taken.is_cuda)
            and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(ctx_lens=ctx_lens, new_lens=new_lens, block_table=block_table, free_blocks=free_blocks,
                              slots=slots, positions=positions, token_to_seq=token_to_seq, cu_new=cu_new,
                              seq_lens=seq_lens, cu_seq=cu_seq, blocks_taken=blocks_taken, error_flag=error_flag)
    words = PLAN_ARGS.pack(
        ctx_lens.data_ptr(), new_lens.data_ptr(), r, block_table.data_ptr(), width,
        free_blocks.data_ptr(), free, num_blocks, block_size, 0 if slots is None else slots.data_ptr(),
        0 if positions is None else positions.data_ptr(), 0 if token_to_seq is None else token_to_seq.data_ptr(), tokens,
        cu_new.data_ptr(), seq_lens.data_ptr(), 0 if cu_seq is None else cu_seq.data_ptr(), taken, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0)
    st = load_library().pmg_call_packed(0, words) if _one_device else _call(0, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_plan_step")


def append(c_kv: torch.Tensor, k_pe: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor,
           cos_sin: torch.Tensor, norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
           scale: Optional[torch.Tensor] = None, q_pe: Optional[torch.Tensor] = None,
           q_out: Optional[torch.Tensor] = None, interleaved: bool = False,
           error_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Norm, rotate and write the entries of new tokens into the paged cache,
    and rotate their queries (pmg_append).

    c_kv [tokens, latent], k_pe [tokens, rope] and q_pe [tokens, heads, rope]
    (bf16, fp16 or fp32, any row strides); cache [num_blocks, block_size,
    latent + rope] (bf16, fp16, fp32 or e4m3 with `scale`); slots int64 and
    positions int32 [tokens] as plan_step writes them; cos_sin fp32
    [num_positions, rope] (cosines, then sines); norm_weight fp32 [latent] or
    None (no norm). q_out like q_pe (it may be q_pe). interleaved: pairs are
    neighbours instead of halves apart.
    """
    shape, cs, kshape, ks, bshape, bs = c_kv.shape, c_kv.stride(), k_pe.shape, k_pe.stride(), cache.shape, cache.stride()
    if not (len(cs) == 2 and len(ks) == 2 and len(bs) == 3 and cs[1] == 1 and ks[1] == 1 and bs[2] == 1):
        _unit_last("c_kv", 2, c_kv)
        _unit_last("k_pe", 2, k_pe)
        _unit_last("cache", 3, cache)
    (t, dv), (tk, dr), (blocks, block_size, entry) = shape, kshape, bshape
    dtype = c_kv.dtype
    src, dst = TORCH_DTYPE_CODES.get(dtype), TORCH_DTYPE_CODES.get(cache.dtype)
    if tk != t or entry != dv + dr:
        raise ValueError(f"c_kv {list(c_kv.shape)}, k_pe {list(k_pe.shape)} and cache {list(cache.shape)} do not fit")
    if src is None or dst is None or k_pe.dtype is not dtype:
        raise ValueError(f"unsupported dtypes {dtype}, {k_pe.dtype} -> {cache.dtype}")
    rot = cos_sin.shape
    if cos_sin.dtype is not _F32 or len(rot) != 2 or rot[1] != dr or not cos_sin.is_contiguous():
        raise ValueError(f"cos_sin must be float32 [num_positions, {dr}] and contiguous")
    if not (slots.dtype is _I64 and slots.numel() == t and slots.is_contiguous()
            and positions.dtype is _I32 and positions.numel() == t and positions.is_contiguous()
            and (norm_weight is None or _is_vector(norm_weight, _F32, dv))):
        _vector(slots, _I64, t, "slots")
        _vector(positions, _I32, t, "positions")
        _vector(norm_weight, _F32, dv, "norm_weight", True)
    if (q_pe is None) != (q_out is None):
        raise ValueError("q_pe and q_out go together")
    q = o = heads = 0
    qs = os_ = (0, 0)
    if q_pe is not None:
        shape, qs, oshape, os_ = q_pe.shape, q_pe.stride(), q_out.shape, q_out.stride()
        if not (len(qs) == 3 and len(os_) == 3 and qs[2] == 1 and os_[2] == 1):
            _unit_last("q_pe", 3, q_pe)
            _unit_last("q_out", 3, q_out)
        heads = shape[1]
        if oshape != shape or shape[0] != t or shape[2] != dr or q_pe.dtype is not dtype or q_out.dtype is not dtype:
            raise ValueError(f"q_pe {list(shape)} and q_out {list(oshape)} must be [{t}, heads, {dr}] of {dtype}")
        q, o = q_pe.data_ptr(), q_out.data_ptr()
    factor, flag = _scalar(scale, _F32, "scale"), _scalar(error_flag, _I32, "error_flag")
    device = 0
    if not (_one_device and c_kv.is_cuda and k_pe.is_cuda and cache.is_cuda and slots.is_cuda and positions.is_cuda
            and cos_sin.is_cuda and (norm_weight is None or norm_weight.is_cuda) and (scale is None or scale.is_cuda)
            and (q_pe is None or q_pe.is_cuda and q_out.is_cuda) and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(c_kv=c_kv, k_pe=k_pe, cache=cache, slots=slots, positions=positions, cos_sin=cos_sin,
                              norm_weight=norm_weight, scale=scale, q_pe=q_pe, q_out=q_out, error_flag=error_flag)
    words = APPEND_ARGS.pack(
        c_kv.data_ptr(), cs[0], k_pe.data_ptr(), ks[0], 0 if norm_weight is None else norm_weight.data_ptr(), eps,
        cos_sin.data_ptr(), rot[0],
        slots.data_ptr(), positions.data_ptr(), t, dv, dr, src, cache.data_ptr(), bs[0], bs[1], blocks, block_size, dst,
        factor, q, qs[0], qs[1], o, os_[0], os_[1], heads, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0, OPT_ROPE_PAIRS if interleaved else 0)
    st = load_library().pmg_call_packed(1, words) if _one_device else _call(1, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_append")


def attention_workspace_bytes() -> int:
    """Bytes of the workspace of latent_decode and latent_prefill on the
    current device, for any sizes."""
    n = load_library().pmg_attention_workspace()
    if n < 0:
        raise PmgError(6, "pmg_attention_workspace")
    return int(n)


def new_attention_workspace(device) -> torch.Tensor:
    """A workspace for latent_decode and latent_prefill. One per stream: calls
    that may overlap must not share one."""
    with torch.cuda.device(device):
        return torch.empty(attention_workspace_bytes(), dtype=torch.uint8, device=device)


def latent_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  out: torch.Tensor, lse: Optional[torch.Tensor] = None, *, sm_scale: float,
                  scale: Optional[torch.Tensor] = None, workspace: torch.Tensor,
                  error_flag: Optional[torch.Tensor] = None, stream=None, options: int = 0) -> None:
    """Absorbed latent attention of q_len new tokens a request over the paged
    cache (pmg_latent_decode).

    q         [num_reqs, q_len, heads, latent + rope] (bf16, fp16 or fp32)
    cache     [num_blocks, block_size, latent + rope] of q's dtype, or e4m3
              with `scale` (fp32 device scalar); the new tokens are in it
    seq_lens  int32 [num_reqs], lengths with the new tokens: token i of q_len
              sees the first seq_len - q_len + 1 + i entries
    out       [num_reqs, q_len, heads, latent] of q's dtype; its last dimension
              sets what is latent and what is rope
    lse       fp32 [num_reqs, q_len, heads], contiguous, or None
    """
    shape, qs, cshape, bs, oshape, os_ = q.shape, q.stride(), cache.shape, cache.stride(), out.shape, out.stride()
    if not (len(qs) == 4 and len(bs) == 3 and len(os_) == 4 and qs[3] == 1 and bs[2] == 1 and os_[3] == 1):
        _unit_last("q", 4, q)
        _unit_last("cache", 3, cache)
        _unit_last("out", 4, out)
    r, q_len, heads, entry = shape
    blocks, block_size, cached = cshape
    out_r, out_len, out_heads, dv = oshape
    if out_r != r or out_len != q_len or out_heads != heads or cached != entry or not 1 <= dv <= entry:
        raise ValueError(f"q {list(shape)}, cache {list(cshape)} and out {list(oshape)} do not fit")
    qd, cd = TORCH_DTYPE_CODES.get(q.dtype), TORCH_DTYPE_CODES.get(cache.dtype)
    if qd is None or cd is None or out.dtype is not q.dtype:
        raise ValueError(f"unsupported dtypes {q.dtype}, {cache.dtype} -> {out.dtype}")
    if not (seq_lens.dtype is _I32 and seq_lens.numel() == r and seq_lens.is_contiguous()
            and (lse is None or lse.dtype is _F32 and lse.numel() == r * q_len * heads and lse.is_contiguous())):
        _vector(seq_lens, _I32, r, "seq_lens")
        _vector(lse, _F32, r * q_len * heads, "lse", True)
    width, factor = _table(block_table, r), 0 if scale is None else _scalar(scale, _F32, "scale")
    flag = 0 if error_flag is None else _scalar(error_flag, _I32, "error_flag")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    device = 0
    if not (_one_device and q.is_cuda and cache.is_cuda and block_table.is_cuda and seq_lens.is_cuda and out.is_cuda
            and workspace.is_cuda and (lse is None or lse.is_cuda) and (scale is None or scale.is_cuda)
            and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(q=q, cache=cache, block_table=block_table, seq_lens=seq_lens, out=out, workspace=workspace,
                              lse=lse, scale=scale, error_flag=error_flag)
    words = DECODE_ARGS.pack(
        q.data_ptr(), qs[0], qs[1], qs[2], cache.data_ptr(), bs[0], bs[1], blocks, block_table.data_ptr(), width,
        seq_lens.data_ptr(), r, q_len, heads, dv, entry - dv, block_size, qd, cd, factor, sm_scale, out.data_ptr(),
        os_[0], os_[1], os_[2], 0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0, options)
    st = load_library().pmg_call_packed(2, words) if _one_device else _call(2, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_latent_decode")


def latent_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                   cu_k: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor] = None, *, sm_scale: float,
                   causal: bool = False, prev_out: Optional[torch.Tensor] = None,
                   prev_lse: Optional[torch.Tensor] = None, workspace: torch.Tensor,
                   error_flag: Optional[torch.Tensor] = None, stream=None, options: int = 0) -> None:
    """Expanded latent attention of a chunk of new tokens (pmg_latent_prefill).

    q       [total_q, heads, nope + rope]; k_nope [total_k, heads, nope]; k_pe
            [total_k, rope], shared by the heads; v [total_k, heads, v_dim];
            out [total_q, heads, v_dim]: one dtype (bf16, fp16 or fp32), any
            strides but the last. Views of one up-projection and of gathered
            entries are taken as they are.
    cu_q, cu_k  int32 [num_reqs + 1]: rows of each request.
    causal  query i of q_len sees the first k_len - q_len + i + 1 keys.
    lse     fp32 [total_q, heads], contiguous, or None.
    prev_out, prev_lse  the result over other keys, joined with this one's
            (they may be out and lse).
    """
    (tq, heads, dk), qs = _unit_last("q", 3, q)
    (tk, kh, dn), ks = _unit_last("k_nope", 3, k_nope)
    (tp, dr), ps = _unit_last("k_pe", 2, k_pe)
    (tv, vh, dv), vs = _unit_last("v", 3, v)
    oshape, os_ = _unit_last("out", 3, out)
    if kh != heads or vh != heads or tv != tk or tp != tk or dn + dr != dk or oshape != (tq, heads, dv):
        raise ValueError(f"q {list(q.shape)}, k_nope {list(k_nope.shape)}, k_pe {list(k_pe.shape)}, v "
                         f"{list(v.shape)} and out {list(oshape)} do not fit")
    dtype = q.dtype
    code = TORCH_DTYPE_CODES.get(dtype)
    if code is None or not (k_nope.dtype is dtype and k_pe.dtype is dtype and v.dtype is dtype and out.dtype is dtype):
        raise ValueError("q, k_nope, k_pe, v and out must have one supported dtype")
    if (prev_out is None) != (prev_lse is None):
        raise ValueError("prev_out and prev_lse go together")
    prev, rs = 0, (0, 0)
    if prev_out is not None:
        pshape, rs = _unit_last("prev_out", 3, prev_out)
        if pshape != oshape or prev_out.dtype is not dtype:
            raise ValueError("prev_out must be like out")
        prev = prev_out.data_ptr()
    reqs = cu_q.numel() - 1
    if not (_is_vector(cu_q, _I32, reqs + 1) and _is_vector(cu_k, _I32, reqs + 1)
            and (lse is None or _is_vector(lse, _F32, tq * heads))
            and (prev_lse is None or _is_vector(prev_lse, _F32, tq * heads))):
        _vector(cu_q, _I32, reqs + 1, "cu_q")
        _vector(cu_k, _I32, reqs + 1, "cu_k")
        _vector(lse, _F32, tq * heads, "lse", True)
        _vector(prev_lse, _F32, tq * heads, "prev_lse", True)
    flag = _scalar(error_flag, _I32, "error_flag")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    device = 0
    if not (_one_device and q.is_cuda and k_nope.is_cuda and k_pe.is_cuda and v.is_cuda and cu_q.is_cuda and cu_k.is_cuda
            and out.is_cuda and workspace.is_cuda and (lse is None or lse.is_cuda)
            and (prev_out is None or prev_out.is_cuda and prev_lse.is_cuda) and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(q=q, k_nope=k_nope, k_pe=k_pe, v=v, cu_q=cu_q, cu_k=cu_k, out=out, workspace=workspace,
                              lse=lse, prev_out=prev_out, prev_lse=prev_lse, error_flag=error_flag)
    words = PREFILL_ARGS.pack(
        q.data_ptr(), qs[0], qs[1], k_nope.data_ptr(), ks[0], ks[1], k_pe.data_ptr(), ps[0], v.data_ptr(), vs[0], vs[1],
        cu_q.data_ptr(), cu_k.data_ptr(), reqs, tq, tk, heads, dn, dr, dv, code, sm_scale, out.data_ptr(), os_[0], os_[1],
        0 if lse is None else lse.data_ptr(), prev, rs[0], rs[1], 0 if prev_lse is None else prev_lse.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0, (OPT_CAUSAL if causal else 0) | options)
    st = load_library().pmg_call_packed(3, words) if _one_device else _call(3, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_latent_prefill")


# --- long contexts (include/pmg_long.h) ------------------------------------------


def block_bounds(cache: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 ctx_lens: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """Largest and smallest value of each column of the pages that entries
    joined (pmg_block_bounds).

    cache     [num_blocks, block_size, entry] (bf16, fp16, fp32 or e4m3)
    bounds    [num_blocks, 2, entry]: largest, then smallest; of cache's dtype, or
              for an e4m3 cache of the queries' (its values without the scale).
              Pages behind each other, or all largest before all smallest
    ctx_lens  int32 [num_reqs]: places that bounds knows of already, or None
    seq_lens  int32 [num_reqs]: places up to which it shall know. plan_step has
              both: one call a step, after append.
    """
    shape, cs, bshape, bs = cache.shape, cache.stride(), bounds.shape, bounds.stride()
    if not (len(cs) == 3 and len(bs) == 3 and cs[2] == 1 and bs[2] == 1):
        _unit_last("cache", 3, cache)
        _unit_last("bounds", 3, bounds)
    blocks, block_size, entry = shape
    if bshape != (blocks, 2, entry):
        raise ValueError(f"bounds {list(bshape)} must be [{blocks}, 2, {entry}]")
    cd, bd = TORCH_DTYPE_CODES.get(cache.dtype), TORCH_DTYPE_CODES.get(bounds.dtype)
    if cd is None or bd is None:
        raise ValueError(f"unsupported dtypes {cache.dtype} -> {bounds.dtype}")
    r = seq_lens.numel()
    if not (seq_lens.dtype is _I32 and seq_lens.is_contiguous()
            and (ctx_lens is None or ctx_lens.dtype is _I32 and ctx_lens.numel() == r and ctx_lens.is_contiguous())):
        _vector(seq_lens, _I32, r, "seq_lens")
        _vector(ctx_lens, _I32, r, "ctx_lens", True)
    width, flag = _table(block_table, r), 0 if error_flag is None else _scalar(error_flag, _I32, "error_flag")
    device = 0
    if not (_one_device and cache.is_cuda and bounds.is_cuda and block_table.is_cuda and seq_lens.is_cuda
            and (ctx_lens is None or ctx_lens.is_cuda) and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(cache=cache, bounds=bounds, block_table=block_table, seq_lens=seq_lens, ctx_lens=ctx_lens,
                              error_flag=error_flag)
    words = BOUNDS_ARGS.pack(
        cache.data_ptr(), cs[0], cs[1], blocks, block_size, entry, cd, bounds.data_ptr(), bs[0], bs[1], bd,
        block_table.data_ptr(), width, 0 if ctx_lens is None else ctx_lens.data_ptr(), seq_lens.data_ptr(), r, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0)
    st = load_library().pmg_call_packed(4, words) if _one_device else _call(4, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_block_bounds")


def _token_rows(what: str, scores: torch.Tensor) -> int:
    """The stride of [num_reqs, q_len, width] scores as num_reqs * q_len rows."""
    (r, n, width), s = _unit_last(what, 3, scores)
    if r > 1 and n > 1 and s[0] != n * s[1]:
        raise ValueError(f"{what}' rows must lie at one stride")
    step = s[1] if n > 1 else s[0] if r > 1 else width
    return max(step, width) if r * n <= 1 else step


def block_scores(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 scores: torch.Tensor, *, block_size: int, sm_scale: float, scale: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None, stream=None,
                 options: int = 0) -> None:
    """The most that entries of each page can score for each new token, over the
    heads (pmg_block_scores).

    q         [num_reqs, q_len, heads, entry] (bf16, fp16 or fp32), as for
              latent_decode
    bounds    [num_blocks, 2, entry] of q's dtype, as block_bounds keeps them
    seq_lens  int32 [num_reqs], lengths with the new tokens
    scores    fp32 [num_reqs, q_len, width of block_table]; -inf for pages of
              which a token sees nothing
    scale     fp32 device scalar of an e4m3 cache, or None
    lse       fp32 [num_reqs, q_len, heads], contiguous, or None: subtracted from
              a head's scores; the log sums of an earlier step make them bounds of
              the logarithms of weights, comparable over the heads
    """
    shape, qs, bshape, bs = q.shape, q.stride(), bounds.shape, bounds.stride()
    if not (len(qs) == 4 and len(bs) == 3 and qs[3] == 1 and bs[2] == 1):
        _unit_last("q", 4, q)
        _unit_last("bounds", 3, bounds)
    r, q_len, heads, entry = shape
    blocks = bshape[0]
    if bshape[1] != 2 or bshape[2] != entry:
        raise ValueError(f"q {list(shape)} and bounds {list(bshape)} do not fit")
    code = TORCH_DTYPE_CODES.get(q.dtype)
    if code is None or bounds.dtype is not q.dtype or scores.dtype is not _F32:
        raise ValueError(f"unsupported dtypes {q.dtype}, {bounds.dtype} -> {scores.dtype}")
    if not (seq_lens.dtype is _I32 and seq_lens.numel() == r and seq_lens.is_contiguous()
            and (lse is None or lse.dtype is _F32 and lse.numel() == r * q_len * heads and lse.is_contiguous())):
        _vector(seq_lens, _I32, r, "seq_lens")
        _vector(lse, _F32, r * q_len * heads, "lse", True)
    width, factor = _table(block_table, r), 0 if scale is None else _scalar(scale, _F32, "scale")
    if scores.shape != (r, q_len, width):
        raise ValueError(f"scores {list(scores.shape)} must be [{r}, {q_len}, {width}]")
    cs = scores.stride()
    if cs[2] != 1:
        _unit_last("scores", 3, scores)
    step = cs[0] if q_len == 1 and r > 1 else _token_rows("scores", scores)
    flag = 0 if error_flag is None else _scalar(error_flag, _I32, "error_flag")
    device = 0
    if not (_one_device and q.is_cuda and bounds.is_cuda and block_table.is_cuda and seq_lens.is_cuda and scores.is_cuda
            and (scale is None or scale.is_cuda) and (lse is None or lse.is_cuda)
            and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(q=q, bounds=bounds, block_table=block_table, seq_lens=seq_lens, scores=scores, scale=scale,
                              lse=lse, error_flag=error_flag)
    words = SCORES_ARGS.pack(
        q.data_ptr(), qs[0], qs[1], qs[2], bounds.data_ptr(), bs[0], bs[1], blocks, block_table.data_ptr(), width,
        seq_lens.data_ptr(), r, q_len, heads, entry, block_size, code, factor, sm_scale,
        0 if lse is None else lse.data_ptr(), scores.data_ptr(), step, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0, options)
    st = load_library().pmg_call_packed(5, words) if _one_device else _call(5, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_block_scores")


def select_blocks(scores: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, selected: torch.Tensor,
                  selected_lens: torch.Tensor, *, block_size: int, first: int = 1, last: int = 1,
                  columns: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """The pages that each new token attends to (pmg_select_blocks): its first
    and last ones and those with the largest scores, selected.shape[1] in all.

    scores         fp32 [num_reqs, q_len, width of block_table]
    selected       int32 [num_reqs * q_len, keep]: their ids in the order of
                   their columns, -1 behind the last
    selected_lens  int32 [num_reqs * q_len]: entries on them that the token sees
    columns        like selected, or None: their columns
    latent_decode(q.view(-1, 1, heads, entry), cache, selected, selected_lens,
    ...) attends to them.
    """
    shape, cs, sshape, ss = scores.shape, scores.stride(), selected.shape, selected.stride()
    if not (len(cs) == 3 and len(ss) == 2 and cs[2] == 1 and ss[1] == 1):
        _unit_last("scores", 3, scores)
        _unit_last("selected", 2, selected)
    (r, q_len, width), (tokens, keep) = shape, sshape
    if scores.dtype is not _F32 or selected.dtype is not _I32:
        raise ValueError(f"scores must be float32 and selected int32, got {scores.dtype} and {selected.dtype}")
    if tokens != r * q_len or _table(block_table, r) != width:
        raise ValueError(f"scores {list(scores.shape)}, block_table {list(block_table.shape)} and selected "
                         f"{list(selected.shape)} do not fit")
    if not (seq_lens.dtype is _I32 and seq_lens.numel() == r and seq_lens.is_contiguous()
            and selected_lens.dtype is _I32 and selected_lens.numel() == tokens and selected_lens.is_contiguous()):
        _vector(seq_lens, _I32, r, "seq_lens")
        _vector(selected_lens, _I32, tokens, "selected_lens")
    if columns is not None and (columns.dtype is not _I32 or columns.shape != selected.shape
                                or columns.stride() != selected.stride()):
        raise ValueError("columns must be like selected")
    step = cs[0] if q_len == 1 and r > 1 else _token_rows("scores", scores)
    flag = 0 if error_flag is None else _scalar(error_flag, _I32, "error_flag")
    device = 0
    if not (_one_device and scores.is_cuda and block_table.is_cuda and seq_lens.is_cuda and selected.is_cuda
            and selected_lens.is_cuda and (columns is None or columns.is_cuda)
            and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(scores=scores, block_table=block_table, seq_lens=seq_lens, selected=selected,
                              selected_lens=selected_lens, columns=columns, error_flag=error_flag)
    words = SELECT_ARGS.pack(
        scores.data_ptr(), step, block_table.data_ptr(), width, seq_lens.data_ptr(), r, q_len, block_size,
        selected.data_ptr(), ss[0] if tokens > 1 else keep, 0 if columns is None else columns.data_ptr(),
        selected_lens.data_ptr(), keep, first, last, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0)
    st = load_library().pmg_call_packed(6, words) if _one_device else _call(6, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_select_blocks")


def shared_workspace_bytes(num_reqs: int, q_len: int, heads: int, latent: int) -> int:
    """Bytes of the workspace of latent_decode_shared for so many rows on the
    current device; enough for any fewer, and for the other attention calls."""
    n = load_library().pmg_shared_workspace(num_reqs * q_len * heads, latent)
    if n < 0:
        raise PmgError(2, "pmg_shared_workspace")
    return int(n)


def new_shared_workspace(device, num_reqs: int, q_len: int, heads: int, latent: int) -> torch.Tensor:
    """A workspace for latent_decode_shared of at most so many rows. One per
    stream: calls that may overlap must not share one."""
    with torch.cuda.device(device):
        return torch.empty(shared_workspace_bytes(num_reqs, q_len, heads, latent), dtype=torch.uint8, device=device)


def latent_decode_shared(q: torch.Tensor, cache: torch.Tensor, prefix_table: torch.Tensor, prefix_lens: torch.Tensor,
                         cu_groups: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                         lse: Optional[torch.Tensor] = None, *, sm_scale: float,
                         scale: Optional[torch.Tensor] = None, workspace: torch.Tensor,
                         error_flag: Optional[torch.Tensor] = None, stream=None, options: int = 0) -> None:
    """Absorbed latent attention of requests behind prefixes that they share
    (pmg_latent_decode_shared).

    prefix_table  int32 [num_groups, width], prefix_lens int32 [num_groups]: pages
                  and lengths of the prefixes
    cu_groups     int32 [num_groups + 1]: requests [cu_groups[g], cu_groups[g + 1])
                  see prefix g; requests of no group see none
    block_table   int32 [num_reqs, width'], seq_lens int32 [num_reqs]: the entries
                  of each request's own, behind its prefix, as in latent_decode
    workspace     new_shared_workspace(device, num_reqs, q_len, heads, latent)
    The rest as in latent_decode.
    """
    shape, qs, cshape, bs, oshape, os_ = q.shape, q.stride(), cache.shape, cache.stride(), out.shape, out.stride()
    if not (len(qs) == 4 and len(bs) == 3 and len(os_) == 4 and qs[3] == 1 and bs[2] == 1 and os_[3] == 1):
        _unit_last("q", 4, q)
        _unit_last("cache", 3, cache)
        _unit_last("out", 4, out)
    r, q_len, heads, entry = shape
    blocks, block_size, cached = cshape
    out_r, out_len, out_heads, dv = oshape
    if out_r != r or out_len != q_len or out_heads != heads or cached != entry or not 1 <= dv <= entry:
        raise ValueError(f"q {list(shape)}, cache {list(cshape)} and out {list(oshape)} do not fit")
    qd, cd = TORCH_DTYPE_CODES.get(q.dtype), TORCH_DTYPE_CODES.get(cache.dtype)
    if qd is None or cd is None or out.dtype is not q.dtype:
        raise ValueError(f"unsupported dtypes {q.dtype}, {cache.dtype} -> {out.dtype}")
    g = prefix_lens.numel()
    if not (_is_vector(seq_lens, _I32, r) and _is_vector(prefix_lens, _I32, g) and _is_vector(cu_groups, _I32, g + 1)
            and (lse is None or _is_vector(lse, _F32, r * q_len * heads))):
        _vector(seq_lens, _I32, r, "seq_lens")
        _vector(prefix_lens, _I32, g, "prefix_lens")
        _vector(cu_groups, _I32, g + 1, "cu_groups")
        _vector(lse, _F32, r * q_len * heads, "lse", True)
    prefix_width, width, factor = _table(prefix_table, g), _table(block_table, r), _scalar(scale, _F32, "scale")
    flag = _scalar(error_flag, _I32, "error_flag")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    device = 0
    if not (_one_device and q.is_cuda and cache.is_cuda and prefix_table.is_cuda and prefix_lens.is_cuda
            and cu_groups.is_cuda and block_table.is_cuda and seq_lens.is_cuda and out.is_cuda and workspace.is_cuda
            and (lse is None or lse.is_cuda) and (scale is None or scale.is_cuda)
            and (error_flag is None or error_flag.is_cuda)):
        device = _same_device(q=q, cache=cache, prefix_table=prefix_table, prefix_lens=prefix_lens, cu_groups=cu_groups,
                              block_table=block_table, seq_lens=seq_lens, out=out, workspace=workspace, lse=lse,
                              scale=scale, error_flag=error_flag)
    words = SHARED_ARGS.pack(
        q.data_ptr(), qs[0], qs[1], qs[2], cache.data_ptr(), bs[0], bs[1], blocks, prefix_table.data_ptr(), prefix_width,
        prefix_lens.data_ptr(), cu_groups.data_ptr(), g, block_table.data_ptr(), width, seq_lens.data_ptr(), r, q_len,
        heads, dv, entry - dv, block_size, qd, cd, factor, sm_scale, out.data_ptr(), os_[0], os_[1], os_[2],
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, flag,
        _raw_stream(device) if stream is None else _stream_handle(stream) or 0, options)
    st = load_library().pmg_call_packed(7, words) if _one_device else _call(7, words, device)
    if st != PMG_OK:
        raise PmgError(st, "pmg_latent_decode_shared")

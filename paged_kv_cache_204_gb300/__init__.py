"""Python binding of the paged KV-cache library (C ABI in include/pkv.h).

Argument marshalling only: every entry point forwards device pointers, sizes
and the current CUDA stream to the compiled library, which does all the work
in its own kernels. There is no fallback: importing this package without the
built library (``python -m paged_kv_cache_204_gb300.build`` or
``__graft_entry__.build()``) raises ImportError.

Functions mirror the C entry points:
  reshape_and_cache       -> pkv_reshape_and_cache
  copy_blocks             -> pkv_copy_blocks
  paged_attention_decode  -> pkv_paged_attention_decode
  decode_workspace_bytes  -> pkv_decode_workspace_bytes
  paged_attention_decode_grouped  -> pkv_paged_attention_decode_grouped
  reshape_and_cache_fp8, paged_attention_decode_fp8  -> the fp8 (e4m3) cache entry points
  reshape_and_cache_q4_0, paged_attention_decode_q4_0, copy_blocks_q4_0
                          -> the 4-bit (q4_0) cache entry points
  paged_attention_prefill -> pkv_paged_attention_prefill
  decode_grouped_workspace_bytes  -> pkv_decode_grouped_workspace_bytes
  paged_attention_decode_window, paged_attention_prefill_window
                          -> attention over the first tokens and a sliding window
  paged_attention_decode_scores, evict_tokens
                          -> decode that adds up attention weights, and the eviction that goes by them
  set_wait_timeout_ns / get_wait_timeout_ns, status_string, version
The host block manager (include/pkv_block_manager.h) is wrapped by
``paged_kv_cache_204_gb300.block_manager.BlockManager``.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

LIB_PATH = _build.LIB

if not os.path.exists(LIB_PATH):
    raise ImportError(f"paged_kv_cache_204_gb300: compiled library missing at {LIB_PATH}; "
                      "build it with `python -m paged_kv_cache_204_gb300.build`")

lib = ctypes.CDLL(LIB_PATH)

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA, PKV_ERR_OUT_OF_BLOCKS = range(6)
DEV_ERR_BLOCK_ID, DEV_ERR_SLOT, DEV_ERR_CONTEXT_LEN, DEV_ERR_TIMEOUT, DEV_ERR_PAIR = 1, 2, 4, 8, 16
DEV_ERR_GROUP = 32
DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.uint8: 3}  # uint8: e4m3 codes
PKV_FP8_E4M3 = 3
PKV_Q4_0 = 4

_P, _I, _I64, _U64, _F, _SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                               ctypes.c_float, ctypes.c_size_t)
lib.pkv_status_string.argtypes = [_I]
lib.pkv_status_string.restype = ctypes.c_char_p
lib.pkv_version.argtypes = []
lib.pkv_version.restype = _I
lib.pkv_set_wait_timeout_ns.argtypes = [_U64]
lib.pkv_set_wait_timeout_ns.restype = None
lib.pkv_get_wait_timeout_ns.argtypes = []
lib.pkv_get_wait_timeout_ns.restype = _U64
lib.pkv_decode_workspace_bytes.argtypes = [_I, _I, _I, _I]
lib.pkv_decode_workspace_bytes.restype = _SZ
lib.pkv_reshape_and_cache.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]
lib.pkv_reshape_and_cache.restype = _I
lib.pkv_copy_blocks.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]
lib.pkv_copy_blocks.restype = _I
lib.pkv_paged_attention_decode.argtypes = [_P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I,
                                           _I, _I, _P, _SZ, _P, _P]
lib.pkv_paged_attention_decode.restype = _I
lib.pkv_paged_attention_decode_grouped.argtypes = [_P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I,
                                                   _I, _I, _P, _P, _I, _I, _P, _SZ, _P, _P]
lib.pkv_paged_attention_decode_grouped.restype = _I
lib.pkv_decode_grouped_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
lib.pkv_decode_grouped_workspace_bytes.restype = _SZ
lib.pkv_reshape_and_cache_fp8.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _P, _P]
lib.pkv_reshape_and_cache_fp8.restype = _I
lib.pkv_paged_attention_decode_fp8.argtypes = [_P, _P, _P, _P, _P, _P, _F, _F, _F, _I, _I, _I, _I, _I, _I, _I,
                                               _I, _I, _P, _SZ, _P, _P]
lib.pkv_paged_attention_decode_fp8.restype = _I
lib.pkv_reshape_and_cache_q4_0.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]
lib.pkv_reshape_and_cache_q4_0.restype = _I
lib.pkv_paged_attention_decode_q4_0.argtypes = [_P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                                _P, _SZ, _P, _P]
lib.pkv_paged_attention_decode_q4_0.restype = _I
lib.pkv_paged_attention_prefill.argtypes = [_P, _P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                              _P, _P]
lib.pkv_paged_attention_prefill.restype = _I
lib.pkv_paged_attention_decode_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I,
                                                   _I, _I, _I, _P, _P]
lib.pkv_paged_attention_decode_noalloc.restype = _I
lib.pkv_decode_window_workspace_bytes.argtypes = [_I, _I, _I, _I]
lib.pkv_decode_window_workspace_bytes.restype = _SZ
lib.pkv_decode_scores_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
lib.pkv_decode_scores_workspace_bytes.restype = _SZ
lib.pkv_paged_attention_decode_window.argtypes = [_P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                                  _I, _I, _P, _SZ, _P, _P]
lib.pkv_paged_attention_decode_window.restype = _I
lib.pkv_paged_attention_prefill_window.argtypes = [_P, _P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _I,
                                                   _I, _I, _I, _P, _P]
lib.pkv_paged_attention_prefill_window.restype = _I
lib.pkv_paged_attention_decode_scores.argtypes = [_P, _P, _P, _I64, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I,
                                                  _I, _I, _I, _P, _SZ, _P, _P]
lib.pkv_paged_attention_decode_scores.restype = _I
lib.pkv_evict_tokens.argtypes = [_P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                 _I, _I, _P, _P]
lib.pkv_evict_tokens.restype = _I
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # PKV_NOALLOC_SCRATCH_BYTES


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


def status_string(status: int) -> str:
    return lib.pkv_status_string(int(status)).decode()


def version() -> int:
    return lib.pkv_version()


def set_wait_timeout_ns(ns: int) -> None:
    lib.pkv_set_wait_timeout_ns(int(ns))


def get_wait_timeout_ns() -> int:
    return lib.pkv_get_wait_timeout_ns()


def decode_workspace_bytes(num_seqs: int, num_heads: int, head_dim: int, max_context_len: int) -> int:
    return lib.pkv_decode_workspace_bytes(num_seqs, num_heads, head_dim, max_context_len)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(status: int, what: str) -> None:
    if status != PKV_OK:
        raise PkvError(status, what)


def reshape_and_cache(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, dev_err: torch.Tensor | None = None,
                      stream=None) -> None:
    """k, v [T, Hkv, D]; k_cache, v_cache [num_blocks, Hkv, block_size, D];
    slot_mapping int64 [T] (all on the GPU)."""
    T, Hkv, D = k.shape
    nb, _, bs, _ = k_cache.shape
    _check(lib.pkv_reshape_and_cache(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                     T, Hkv, D, bs, nb, DTYPE_CODE[k_cache.dtype], _ptr(dev_err),
                                     _stream(stream)), "pkv_reshape_and_cache")


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_pairs: torch.Tensor,
                dev_err: torch.Tensor | None = None, stream=None) -> None:
    """block_pairs int64 [n, 2] (src, dst) on the GPU."""
    nb, Hkv, bs, D = k_cache.shape
    n = block_pairs.numel() // 2
    _check(lib.pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_pairs), n, Hkv, D, bs, nb,
                               DTYPE_CODE[k_cache.dtype], _ptr(dev_err), _stream(stream)),
           "pkv_copy_blocks")


def paged_attention_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, scale: float, max_context_len: int,
                           workspace: torch.Tensor | None = None,
                           dev_err: torch.Tensor | None = None, stream=None) -> None:
    """out, q [B, H, D]; caches [num_blocks, Hkv, block_size, D]; block_tables
    int32 [B, max_blocks_per_seq]; context_lens int32 [B]; workspace: a
    zero-initialised device buffer of decode_workspace_bytes() bytes (reused
    across calls; the library leaves its counters zero)."""
    B, H, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.pkv_paged_attention_decode(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        float(scale), H, Hkv, D, bs, B, block_tables.shape[1], nb, int(max_context_len),
        DTYPE_CODE[q.dtype], _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream)),
        "pkv_paged_attention_decode")


def paged_attention_decode_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, scale: float, max_context_len: int,
                                   dev_err: torch.Tensor | None = None, stream=None) -> None:
    """paged_attention_decode without a workspace: for callers that cannot
    allocate device memory, the library keeps the partial results of long
    contexts in its own fixed 32 MiB device array (sizes that need more are
    rejected). Calls that overlap on the GPU share that array and race."""
    B, H, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    _check(lib.pkv_paged_attention_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        float(scale), H, Hkv, D, bs, B, block_tables.shape[1], nb, int(max_context_len),
        DTYPE_CODE[q.dtype], _ptr(dev_err), _stream(stream)),
        "pkv_paged_attention_decode_noalloc")


def reshape_and_cache_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                          dev_err: torch.Tensor | None = None, stream=None) -> None:
    """k, v [T, Hkv, D] fp16/bf16; k_cache, v_cache uint8 [num_blocks, Hkv,
    block_size, D] of e4m3 codes; element x is stored as e4m3(x / scale)."""
    T, Hkv, D = k.shape
    nb, _, bs, _ = k_cache.shape
    _check(lib.pkv_reshape_and_cache_fp8(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), T, Hkv,
                                         D, bs, nb, DTYPE_CODE[k.dtype], float(k_scale), float(v_scale), _ptr(dev_err),
                                         _stream(stream)), "pkv_reshape_and_cache_fp8")


def paged_attention_decode_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                               k_scale: float, v_scale: float, max_context_len: int,
                               workspace: torch.Tensor | None = None, dev_err: torch.Tensor | None = None,
                               stream=None) -> None:
    """paged_attention_decode over uint8 pools of e4m3 codes: K values are
    k_scale * code, V values v_scale * code; q, out fp16/bf16."""
    B, H, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.pkv_paged_attention_decode_fp8(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        float(scale), float(k_scale), float(v_scale), H, Hkv, D, bs, B, block_tables.shape[1], nb,
        int(max_context_len), DTYPE_CODE[q.dtype], _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream)),
        "pkv_paged_attention_decode_fp8")


def q4_0_row_bytes(head_dim: int) -> int:
    """Bytes of one q4_0 cache row: head_dim / 32 binary16 scales, then
    head_dim / 2 code bytes."""
    return head_dim // 16 * 9


def reshape_and_cache_q4_0(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           slot_mapping: torch.Tensor, dev_err: torch.Tensor | None = None, stream=None) -> None:
    """k, v [T, Hkv, D] fp16/bf16; k_cache, v_cache uint8 [num_blocks, Hkv,
    block_size, 9 D / 16] of q4_0 rows."""
    T, Hkv, D = k.shape
    nb, _, bs, _ = k_cache.shape
    _check(lib.pkv_reshape_and_cache_q4_0(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), T,
                                          Hkv, D, bs, nb, DTYPE_CODE[k.dtype], _ptr(dev_err), _stream(stream)),
           "pkv_reshape_and_cache_q4_0")


def paged_attention_decode_q4_0(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                                max_context_len: int, workspace: torch.Tensor | None = None,
                                dev_err: torch.Tensor | None = None, stream=None) -> None:
    """paged_attention_decode over uint8 pools of q4_0 rows; q, out fp16/bf16."""
    B, H, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.pkv_paged_attention_decode_q4_0(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        float(scale), H, Hkv, D, bs, B, block_tables.shape[1], nb, int(max_context_len), DTYPE_CODE[q.dtype],
        _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream)), "pkv_paged_attention_decode_q4_0")


def copy_blocks_q4_0(k_cache: torch.Tensor, v_cache: torch.Tensor, block_pairs: torch.Tensor, head_dim: int,
                     dev_err: torch.Tensor | None = None, stream=None) -> None:
    """copy_blocks over uint8 pools of q4_0 rows of head_dim values."""
    nb, Hkv, bs, _ = k_cache.shape
    n = block_pairs.numel() // 2
    _check(lib.pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_pairs), n, Hkv, int(head_dim), bs, nb,
                               PKV_Q4_0, _ptr(dev_err), _stream(stream)), "pkv_copy_blocks")


def paged_attention_prefill(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor,
                            scale: float, max_query_len: int, dev_err: torch.Tensor | None = None,
                            stream=None) -> None:
    """Causal attention of each sequence's last n = query_start[s+1] -
    query_start[s] tokens over its paged context. q, out [total_queries, H, D]
    (fp16/bf16) packed by sequence; query_start int32 [B+1] (on the GPU)."""
    _, H, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    B = context_lens.numel()
    _check(lib.pkv_paged_attention_prefill(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), _ptr(query_start),
        float(scale), H, Hkv, D, bs, B, block_tables.shape[1], nb, int(max_query_len), DTYPE_CODE[q.dtype],
        _ptr(dev_err), _stream(stream)), "pkv_paged_attention_prefill")


def decode_grouped_workspace_bytes(num_seqs: int, num_heads: int, head_dim: int, max_context_len: int,
                                   num_groups: int) -> int:
    return lib.pkv_decode_grouped_workspace_bytes(num_seqs, num_heads, head_dim, max_context_len, num_groups)


def paged_attention_decode_grouped(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, scale: float, max_context_len: int,
                                   group_start: torch.Tensor, shared_blocks: torch.Tensor,
                                   workspace: torch.Tensor, dev_err: torch.Tensor | None = None,
                                   stream=None) -> None:
    """paged_attention_decode for groups of sequences sharing prefix blocks:
    group g = sequences group_start[g]:group_start[g+1] (int32 [G+1]) whose
    first shared_blocks[g] (int32 [G]) block-table entries are the same
    physical blocks. workspace: zero-initialised, decode_grouped_workspace_bytes()."""
    B, H, D = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    G = shared_blocks.numel()
    _check(lib.pkv_paged_attention_decode_grouped(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        float(scale), H, Hkv, D, bs, B, block_tables.shape[1], nb, int(max_context_len),
        _ptr(group_start), _ptr(shared_blocks), G, DTYPE_CODE[q.dtype], _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_err), _stream(stream)),
        "pkv_paged_attention_decode_grouped")


def new_grouped_workspace(num_seqs: int, num_heads: int, head_dim: int, max_context_len: int,
                          num_groups: int, device="cuda") -> torch.Tensor:
    n = decode_grouped_workspace_bytes(num_seqs, num_heads, head_dim, max_context_len, num_groups)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def new_workspace(num_seqs: int, num_heads: int, head_dim: int, max_context_len: int,
                  device="cuda") -> torch.Tensor | None:
    """A zeroed workspace of the size the decode call needs (None if 0)."""
    n = decode_workspace_bytes(num_seqs, num_heads, head_dim, max_context_len)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def decode_window_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return lib.pkv_decode_window_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim)


def decode_scores_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                  max_context_len: int) -> int:
    return lib.pkv_decode_scores_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len)


def new_window_workspace(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                         device="cuda") -> torch.Tensor:
    """A zeroed workspace of paged_attention_decode_window."""
    n = decode_window_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def new_scores_workspace(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, max_context_len: int,
                         device="cuda") -> torch.Tensor:
    """A workspace of paged_attention_decode_scores: its counters zeroed, the
    room for the logits as it comes."""
    n = decode_scores_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:4 * num_seqs * num_heads].zero_()
    return ws


def _want(t: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device, what: str) -> int:
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: need a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _pools(k_cache: torch.Tensor, v_cache: torch.Tensor) -> torch.device:
    """The pools' device, which every other tensor of the call has to be on."""
    dev = k_cache.device
    if dev.type != "cuda":
        raise ValueError(f"k_cache: need a CUDA tensor, got {dev}")
    if k_cache.dim() != 4 or not k_cache.is_contiguous():
        raise ValueError("k_cache: need a contiguous [num_blocks, Hkv, block_size, D] tensor")
    _want(v_cache, k_cache.shape, k_cache.dtype, dev, "v_cache")
    return dev


def _tables(block_tables: torch.Tensor, context_lens: torch.Tensor, dev: torch.device) -> tuple[int, int, int, int]:
    """(sequences, table width, address of the tables, address of the lengths)"""
    if block_tables.dim() != 2:
        raise ValueError("block_tables: need [num_seqs, max_blocks_per_seq]")
    B, MB = block_tables.shape
    return (B, MB, _want(block_tables, (B, MB), torch.int32, dev, "block_tables"),
            _want(context_lens, (B,), torch.int32, dev, "context_lens"))


def _space(workspace: torch.Tensor, dev: torch.device) -> tuple[int, int]:
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: need a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _err_ptr(dev_err: torch.Tensor | None, dev: torch.device) -> int | None:
    if dev_err is None:
        return None
    if dev_err.dtype != torch.int32 or dev_err.numel() < 1 or dev_err.device != dev:
        raise ValueError(f"dev_err: need an int32 tensor on {dev}")
    return dev_err.data_ptr()


def _call(fn, what: str, dev: torch.device, stream, *args) -> None:
    """Call `fn` with the tensors' device current and, unless one is given,
    that device's current stream."""
    if dev.index == torch.cuda.current_device():
        s = torch.cuda.current_stream() if stream is None else stream
        status = fn(*args, s.cuda_stream)
    else:
        with torch.cuda.device(dev):
            s = torch.cuda.current_stream() if stream is None else stream
            status = fn(*args, s.cuda_stream)
    if status != PKV_OK:
        raise PkvError(status, what)


def _code(dtype: torch.dtype, what: str) -> int:
    code = DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError(f"{what}: {dtype} is not a type of this library")
    return code


def paged_attention_decode_window(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, window: int,
                                  num_sinks: int, max_context_len: int, workspace: torch.Tensor,
                                  dev_err: torch.Tensor | None = None, stream=None) -> None:
    """paged_attention_decode in which the query sees its sequence's first
    num_sinks tokens and its newest `window` (the query's own included).
    Block-table entries of blocks with no visible token are not read.
    workspace: new_window_workspace()."""
    dev = _pools(k_cache, v_cache)
    nb, Hkv, bs, D = k_cache.shape
    B, MB, bt, cl = _tables(block_tables, context_lens, dev)
    H = q.shape[1] if q.dim() == 3 else -1
    qp = _want(q, (B, H, D), k_cache.dtype, dev, "q")
    op = _want(out, (B, H, D), k_cache.dtype, dev, "out")
    ws, nbytes = _space(workspace, dev)
    _call(lib.pkv_paged_attention_decode_window, "pkv_paged_attention_decode_window", dev, stream, op, qp,
          k_cache.data_ptr(), v_cache.data_ptr(), bt, cl, scale, window, num_sinks, H, Hkv, D, bs, B, MB, nb,
          max_context_len, _code(q.dtype, "q"), ws, nbytes, _err_ptr(dev_err, dev))


def paged_attention_prefill_window(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_tables: torch.Tensor, context_lens: torch.Tensor,
                                   query_start: torch.Tensor, scale: float, window: int, num_sinks: int,
                                   max_query_len: int, dev_err: torch.Tensor | None = None, stream=None) -> None:
    """paged_attention_prefill in which the query at position P sees the tokens
    t <= P with t < num_sinks or t > P - window."""
    dev = _pools(k_cache, v_cache)
    nb, Hkv, bs, D = k_cache.shape
    B, MB, bt, cl = _tables(block_tables, context_lens, dev)
    N, H = q.shape[:2] if q.dim() == 3 else (-1, -1)
    qp = _want(q, (N, H, D), k_cache.dtype, dev, "q")
    op = _want(out, (N, H, D), k_cache.dtype, dev, "out")
    qs = _want(query_start, (B + 1,), torch.int32, dev, "query_start")
    _call(lib.pkv_paged_attention_prefill_window, "pkv_paged_attention_prefill_window", dev, stream, op, qp,
          k_cache.data_ptr(), v_cache.data_ptr(), bt, cl, qs, scale, window, num_sinks, H, Hkv, D, bs, B, MB, nb,
          max_query_len, _code(q.dtype, "q"), _err_ptr(dev_err, dev))


def _score_rows(t: torch.Tensor, B: int, Hkv: int, dev: torch.device, what: str) -> tuple[int, int]:
    """(address, stride of a row) of a score array [B, Hkv, n]."""
    n = t.shape[2] if t.dim() == 3 else -1
    return _want(t, (B, Hkv, n), torch.float32, dev, what), n


def paged_attention_decode_scores(out: torch.Tensor, scores_out: torch.Tensor, q: torch.Tensor,
                                  k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                                  context_lens: torch.Tensor, scale: float, max_context_len: int,
                                  workspace: torch.Tensor, scores: torch.Tensor | None = None,
                                  dev_err: torch.Tensor | None = None, stream=None) -> None:
    """paged_attention_decode that adds every cached token's attention weight,
    summed over the query heads of its kv head, to its score. scores_out,
    scores float32 [B, Hkv, n >= max_context_len]; scores None: zeros;
    scores_out may be scores (in place). The newest token starts from zero.
    workspace: new_scores_workspace()."""
    dev = _pools(k_cache, v_cache)
    nb, Hkv, bs, D = k_cache.shape
    B, MB, bt, cl = _tables(block_tables, context_lens, dev)
    H = q.shape[1] if q.dim() == 3 else -1
    qp = _want(q, (B, H, D), k_cache.dtype, dev, "q")
    op = _want(out, (B, H, D), k_cache.dtype, dev, "out")
    so, stride = _score_rows(scores_out, B, Hkv, dev, "scores_out")
    si = None if scores is None else _want(scores, scores_out.shape, torch.float32, dev, "scores")
    ws, nbytes = _space(workspace, dev)
    _call(lib.pkv_paged_attention_decode_scores, "pkv_paged_attention_decode_scores", dev, stream, op, so, si, stride,
          qp, k_cache.data_ptr(), v_cache.data_ptr(), bt, cl, scale, H, Hkv, D, bs, B, MB, nb, max_context_len,
          _code(q.dtype, "q"), ws, nbytes, _err_ptr(dev_err, dev))


def evict_tokens(k_cache: torch.Tensor, v_cache: torch.Tensor, scores: torch.Tensor, scores_out: torch.Tensor,
                 block_tables: torch.Tensor, dst_block_tables: torch.Tensor, context_lens: torch.Tensor,
                 new_context_lens: torch.Tensor, kept: torch.Tensor, num_sinks: int, num_recent: int,
                 max_context_len: int, head_dim: int | None = None, dev_err: torch.Tensor | None = None,
                 stream=None) -> None:
    """Cut every sequence to at most budget = kept.shape[2] tokens per kv head:
    its first num_sinks, its last num_recent and the highest-scored between;
    the kept rows of K, V and the scores move up in their order. scores
    float32 [B, Hkv, n]; scores_out likewise (may be scores); kept int32
    [B, Hkv, budget]; new_context_lens may be context_lens. dst_block_tables:
    block_tables itself for sequences that share no block, or a table whose
    blocks are each the same as in block_tables or in no row of it
    (BlockManager.shrink_batch). Pools of any cache type; head_dim for uint8
    pools of q4_0 rows."""
    dev = _pools(k_cache, v_cache)
    nb, Hkv, bs, row = k_cache.shape
    B, MB, bt, cl = _tables(block_tables, context_lens, dev)
    dst = _want(dst_block_tables, (B, MB), torch.int32, dev, "dst_block_tables")
    nl = _want(new_context_lens, (B,), torch.int32, dev, "new_context_lens")
    si, s_in = _score_rows(scores, B, Hkv, dev, "scores")
    so, s_out = _score_rows(scores_out, B, Hkv, dev, "scores_out")
    budget = kept.shape[2] if kept.dim() == 3 else -1
    kp = _want(kept, (B, Hkv, budget), torch.int32, dev, "kept")
    code = _code(k_cache.dtype, "k_cache")
    D = row
    if head_dim is not None and head_dim != row:
        if k_cache.dtype != torch.uint8 or q4_0_row_bytes(head_dim) != row:
            raise ValueError(f"rows of {row} {k_cache.dtype} are no rows of head_dim {head_dim}")
        D, code = head_dim, PKV_Q4_0
    _call(lib.pkv_evict_tokens, "pkv_evict_tokens", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), si, s_in, so,
          s_out, bt, dst, cl, nl, kp, budget, num_sinks, num_recent, Hkv, D, bs, B, MB, nb, max_context_len, code,
          _err_ptr(dev_err, dev))

"""ctypes binding of libdsa_indexer.so: argument marshalling only.

Every computation happens in the library's CUDA kernels.  There is no CPU
fallback: if the shared library is missing, :func:`load` raises.  Tensors are
PyTorch tensors used as device buffers; the binding checks dtypes, devices,
shapes and contiguity, then passes raw pointers and the current CUDA stream.
"""

from __future__ import annotations

import ctypes
import struct
from pathlib import Path
from typing import Optional, Sequence

import torch

LIB_PATH = Path(__file__).resolve().parent / "_lib" / "libdsa_indexer.so"

HEAD_DIM = 128
PAGE_TOKENS = 64
PAGE_BYTES = 8448
PAGE_SCALE_OFFSET = 8192
MAX_TOPK = 2048

DSA_OK = 0
ERRORS = {
    -1: "INVALID_ARG",
    -2: "UNSUPPORTED",
    -3: "WORKSPACE_TOO_SMALL",
    -4: "CUDA",
    -5: "TIMEOUT",
}
STATUS_BAD_PAGE = 0x1
STATUS_BAD_METADATA = 0x2
STATUS_TIMEOUT = 0x4
STATUS_NO_PAGES = 0x8

# every symbol declared in include/dsa_indexer.h
EXPORTS = (
    "dsa_abi_version",
    "dsa_last_error",
    "dsa_last_launch_count",
    "dsa_indexer_write_k",
    "dsa_indexer_write_k_bf16",
    "dsa_indexer_write_k_compressed",
    "dsa_quantize_fp8_blocks",
    "dsa_indexer_workspace_bytes",
    "dsa_indexer_score_topk",
    "dsa_indexer_score_topk_no_alloc",
    "dsa_indexer_score_topk_compressed",
    "dsa_indexer_no_alloc_workspace_bytes",
    "dsa_layer_is_full",
    "dsa_layer_stack_run",
    "dsa_layer_stack_run_bf16",
    "dsa_layer_stack_run_compressed",
    "dsa_mla_write_kv",
    "dsa_sparse_mla_attention",
    "dsa_block_tables_build",
    "dsa_kv_write",
    "dsa_paged_attention_workspace_bytes",
    "dsa_paged_attention",
    "dsa_add_rms_norm",
    "dsa_fp8_matmul",
    "dsa_grouped_matmul",
    "dsa_route_experts",
    "dsa_combine_experts",
)


class DsaError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{ERRORS.get(code, code)}: {message}")
        self.code = code


class LayerIO(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("q_fp8", ctypes.c_void_p),
        ("q_scale", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p),
        ("score_begin", ctypes.c_void_p),
        ("score_end", ctypes.c_void_p),
    ]


class LayerIOBf16(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p),
        ("q_fp8", ctypes.c_void_p),
        ("q_scale", ctypes.c_void_p),
        ("score_begin", ctypes.c_void_p),
        ("score_end", ctypes.c_void_p),
    ]


class KvCache(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
        + [(n, ctypes.c_int64) for n in (
            "k_page_stride", "k_token_stride", "k_head_stride",
            "v_page_stride", "v_token_stride", "v_head_stride",
            "k_scale_page_stride", "k_scale_head_stride",
            "v_scale_page_stride", "v_scale_head_stride", "num_pages")]
        + [(n, ctypes.c_int) for n in ("num_kv_heads", "head_dim", "type")])


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


def _declare(lib: ctypes.CDLL) -> None:
    lib.dsa_abi_version.restype = _I
    lib.dsa_abi_version.argtypes = []
    lib.dsa_last_error.restype = ctypes.c_char_p
    lib.dsa_last_error.argtypes = []
    lib.dsa_last_launch_count.restype = _I
    lib.dsa_last_launch_count.argtypes = []
    lib.dsa_indexer_write_k.restype = _I
    lib.dsa_indexer_write_k.argtypes = [_P, _I, _P, _P, _I, _P, _I, _P, _I64, _P, _P, _P]
    lib.dsa_indexer_write_k_bf16.restype = _I
    lib.dsa_indexer_write_k_bf16.argtypes = [
        _P, _I, _P, _P, _I, _P, _I, _P, _I64, _P, _I, _P, _P, _P, _P, _P]
    lib.dsa_indexer_write_k_compressed.restype = _I
    lib.dsa_indexer_write_k_compressed.argtypes = [
        _P, _I, _P, _P, _I, _P, _I, _P, _I64, _I, _P, _P, _P]
    lib.dsa_quantize_fp8_blocks.restype = _I
    lib.dsa_quantize_fp8_blocks.argtypes = [_P, _I64, _P, _P, _P]
    lib.dsa_indexer_workspace_bytes.restype = _SZ
    lib.dsa_indexer_workspace_bytes.argtypes = [_I, _I, _I, _I64, _I]
    lib.dsa_indexer_score_topk.restype = _I
    lib.dsa_indexer_score_topk.argtypes = [
        _P, _P, _P, _I, _I, _P, _I64, _P, _P, _I, _P, _I, _I, _P, _I, _P, _I64, _P, _SZ, _P, _P]
    lib.dsa_indexer_score_topk_no_alloc.restype = _I
    lib.dsa_indexer_score_topk_no_alloc.argtypes = [
        _P, _P, _P, _I, _I, _P, _I64, _P, _P, _I, _P, _I, _I, _P, _I, _P, _P]
    lib.dsa_indexer_score_topk_compressed.restype = _I
    lib.dsa_indexer_score_topk_compressed.argtypes = [
        _P, _P, _P, _I, _I, _P, _I64, _P, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I64, _P, _SZ, _P,
        _P]
    lib.dsa_indexer_no_alloc_workspace_bytes.restype = _SZ
    lib.dsa_indexer_no_alloc_workspace_bytes.argtypes = []
    lib.dsa_layer_is_full.restype = _I
    lib.dsa_layer_is_full.argtypes = [_I, ctypes.c_char_p, _I, _I]
    lib.dsa_layer_stack_run.restype = _I
    lib.dsa_layer_stack_run.argtypes = [
        _I, ctypes.c_char_p, _I, _I, ctypes.POINTER(LayerIO), _I, _I, _P, _P, _I, _P, _I, _I64,
        _I, _P, _I, ctypes.POINTER(ctypes.c_void_p), _P, _P, _SZ, _P, _P]
    lib.dsa_layer_stack_run_compressed.restype = _I
    lib.dsa_layer_stack_run_compressed.argtypes = [
        _I, ctypes.c_char_p, _I, _I, ctypes.POINTER(LayerIO), _I, _I, _P, _P, _I, _P, _I, _I64,
        _I, _I, _P, _I, ctypes.POINTER(ctypes.c_void_p), _P, _P, _SZ, _P, _P]
    lib.dsa_mla_write_kv.restype = _I
    lib.dsa_mla_write_kv.argtypes = [_P, _I, _P, _P, _I, _P, _I, _P, _I64, _P, _P, _P]
    lib.dsa_sparse_mla_attention.restype = _I
    lib.dsa_sparse_mla_attention.argtypes = [
        _P, _I, _I, _P, _I64, _P, _P, _I, _P, _I, _P, _I, ctypes.c_float, _P, _P, _P, _P]
    _F = ctypes.c_float
    lib.dsa_block_tables_build.restype = _I
    lib.dsa_block_tables_build.argtypes = [_P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P]
    lib.dsa_kv_write.restype = _I
    lib.dsa_kv_write.argtypes = [
        _P, _I64, _I64, _P, _I64, _I64, _I, _I, _P, _P, _P, _P]
    lib.dsa_paged_attention_workspace_bytes.restype = _SZ
    lib.dsa_paged_attention_workspace_bytes.argtypes = []
    lib.dsa_paged_attention.restype = _I
    lib.dsa_paged_attention.argtypes = [
        _P, _I64, _I64, _I, _I, _I, _P, _P, _P, _I, _P, _I, _F, _I, _I, _P,
        _I64, _I64, _P, _P, _SZ, _P, _P]
    lib.dsa_add_rms_norm.restype = _I
    lib.dsa_add_rms_norm.argtypes = [
        _P, _I64, _P, _I64, _P, _I, _I, _I, _F, _P, _I64, _P, _I64, _P, _P, _P]
    lib.dsa_fp8_matmul.restype = _I
    lib.dsa_fp8_matmul.argtypes = [
        _P, _I64, _P, _I, _P, _I64, _P, _I, _I, _I, _P, _I64, _I, _P, _P, _P, _P]
    lib.dsa_grouped_matmul.restype = _I
    lib.dsa_grouped_matmul.argtypes = [
        _P, _I64, _P, _I, _I, _P, _I, _P, _I64, _I64, _P, _I, _I, _P, _I, _I, _P, _I64, _I, _P, _P, _P, _P]
    lib.dsa_route_experts.restype = _I
    lib.dsa_route_experts.argtypes = [
        _P, _I64, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P, _P]
    lib.dsa_combine_experts.restype = _I
    lib.dsa_combine_experts.argtypes = [
        _P, _I64, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P, _I64, _P, _P]
    lib.dsa_layer_stack_run_bf16.restype = _I
    lib.dsa_layer_stack_run_bf16.argtypes = [
        _I, ctypes.c_char_p, _I, _I, ctypes.POINTER(LayerIOBf16), _I, _I, _P, _P, _I, _P, _I,
        _I64, _I, _P, _I, ctypes.POINTER(ctypes.c_void_p), _P, _P, _SZ, _P, _P]


def load() -> ctypes.CDLL:
    """Load the library (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise ImportError(
                f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                "(there is no CPU fallback for the indexer path)")
        lib = ctypes.CDLL(str(LIB_PATH))
        _declare(lib)
        _lib = lib
    return _lib


def _check(rc: int) -> None:
    if rc != DSA_OK:
        msg = load().dsa_last_error().decode(errors="replace")
        raise DsaError(rc, msg)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory for a call's output, of the stream it is launched on: taken for the current one
    it could still be in use there by work that was queued before."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_current_device = torch._C._cuda_getDevice


def _refuse_device(device: int, name: str) -> None:
    raise ValueError(f"{name} lies on cuda:{device}, but cuda:{_current_device()} is the current device, which a call "
                     f"launches on: make it within torch.cuda.device({device})")


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _current_device():
        _refuse_device(t.get_device(), name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None:
        for i, (a, b) in enumerate(zip(t.shape, shape)):
            if b is not None and a != b:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if len(t.shape) != len(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


# ----------------------------------------------------------------------------
# entry points
# ----------------------------------------------------------------------------

def abi_version() -> int:
    return load().dsa_abi_version()


def last_launch_count() -> int:
    return load().dsa_last_launch_count()


def layer_is_full(layer_id: int, pattern: Optional[str] = None, freq: int = 1, offset: int = 2) -> bool:
    rc = load().dsa_layer_is_full(layer_id, None if pattern is None else pattern.encode(), freq, offset)
    if rc < 0:
        _check(rc)
    return bool(rc)


def workspace_bytes(T: int, H: int, R: int, index_topk: int, max_ctx: int = 0) -> int:
    n = load().dsa_indexer_workspace_bytes(T, H, R, max_ctx, index_topk)
    if n == 0:
        raise DsaError(-1, f"no workspace size for T={T}, H={H}, R={R}, index_topk={index_topk}")
    return int(n)


def alloc_workspace(T: int, H: int, R: int, index_topk: int, device="cuda",
                    max_ctx: int = 0) -> torch.Tensor:
    """Workspace for score_topk / layer_stack_run.  0 < max_ctx <= 8192 (a bound on
    the keys any row sees) also makes room for decode rows to be scored into the
    workspace and selected by a second kernel (see dsa_indexer_workspace_bytes)."""
    n = workspace_bytes(T, H, R, index_topk, max_ctx)
    return torch.empty(n, dtype=torch.uint8, device=device)


def quantize_fp8_blocks(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                        scales: Optional[torch.Tensor] = None, stream=None):
    """x [..., 128] FP32 -> (codes uint8 [..., 128], scales FP32 [...])."""
    _need(x, "x", torch.float32)
    if x.shape[-1] != HEAD_DIM:
        raise ValueError("last dimension must be 128")
    nb = x.numel() // HEAD_DIM
    if codes is None:
        codes = _empty(x.shape, torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty(x.shape[:-1], torch.float32, x.device, stream)
    _need(codes, "codes", torch.uint8)
    _need(scales, "scales", torch.float32)
    _check(load().dsa_quantize_fp8_blocks(_ptr(x), nb, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def write_k(k: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
            block_table: torch.Tensor, k_cache: torch.Tensor,
            slot_mapping: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            stream=None) -> None:
    _check(load().dsa_indexer_write_k(*_write_k_args(
        k, query_start_loc, seq_lens, block_table, k_cache, slot_mapping, status, stream)))


def write_k_compressed(k: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                       block_table: torch.Tensor, k_cache: torch.Tensor, compress_ratio: int,
                       slot_mapping: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Cache write into a compressed cache: only tokens with
    (pos + 1) % compress_ratio == 0 are stored, as entry pos // compress_ratio."""
    a = _write_k_args(k, query_start_loc, seq_lens, block_table, k_cache, slot_mapping, status,
                      stream)
    _check(load().dsa_indexer_write_k_compressed(*a[:9], int(compress_ratio), *a[9:]))


def _write_k_args(k, query_start_loc, seq_lens, block_table, k_cache, slot_mapping, status,
                  stream):
    T = k.shape[0]
    R = seq_lens.shape[0]
    _need(k, "k", torch.float32, (T, HEAD_DIM))
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(k_cache, "k_cache", torch.uint8, (None, PAGE_BYTES))
    if slot_mapping is not None:
        _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    if status is not None:
        _need(status, "status", torch.int32)
    return (_ptr(k), T, _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table),
            block_table.shape[1], _ptr(k_cache), k_cache.shape[0], _ptr(slot_mapping),
            _ptr(status), _stream(stream))


def write_k_bf16(k: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                 block_table: torch.Tensor, k_cache: torch.Tensor,
                 q: Optional[torch.Tensor] = None, q_fp8: Optional[torch.Tensor] = None,
                 q_scale: Optional[torch.Tensor] = None,
                 slot_mapping: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Cache write of BF16 keys; with ``q`` [T, H, 128] BF16 the same launch
    quantises the query rows into ``q_fp8`` [T, H, 128] uint8 and ``q_scale``
    [T, H] float32."""
    T = k.shape[0]
    R = seq_lens.shape[0]
    _need(k, "k", torch.bfloat16, (T, HEAD_DIM))
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(k_cache, "k_cache", torch.uint8, (None, PAGE_BYTES))
    H = 0
    if q is not None:
        H = q.shape[1]
        _need(q, "q", torch.bfloat16, (T, H, HEAD_DIM))
        _need(q_fp8, "q_fp8", torch.uint8, (T, H, HEAD_DIM))
        _need(q_scale, "q_scale", torch.float32, (T, H))
    if slot_mapping is not None:
        _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    if status is not None:
        _need(status, "status", torch.int32)
    _check(load().dsa_indexer_write_k_bf16(
        _ptr(k), T, _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table),
        block_table.shape[1], _ptr(k_cache), k_cache.shape[0], _ptr(q), H, _ptr(q_fp8),
        _ptr(q_scale), _ptr(slot_mapping), _ptr(status), _stream(stream)))


def score_topk(q_fp8: torch.Tensor, q_scale: torch.Tensor, w: torch.Tensor,
               k_cache: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
               block_table: torch.Tensor, index_topk: int, topk_buffer: torch.Tensor,
               workspace: torch.Tensor, scores_out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> None:
    _check(load().dsa_indexer_score_topk(*_score_args(
        q_fp8, q_scale, w, k_cache, query_start_loc, seq_lens, block_table, index_topk,
        topk_buffer, workspace, scores_out, status, stream)))


def score_topk_compressed(q_fp8: torch.Tensor, q_scale: torch.Tensor, w: torch.Tensor,
                          k_cache: torch.Tensor, query_start_loc: torch.Tensor,
                          seq_lens: torch.Tensor, block_table: torch.Tensor, compress_ratio: int,
                          index_topk: int, topk_buffer: torch.Tensor, workspace: torch.Tensor,
                          scores_out: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream=None) -> None:
    """score_topk over a compressed cache: row t ranks the entries
    c < (pos + 1) // compress_ratio; indices (and scores_out columns) are entries."""
    a = _score_args(q_fp8, q_scale, w, k_cache, query_start_loc, seq_lens, block_table,
                    index_topk, topk_buffer, workspace, scores_out, status, stream)
    _check(load().dsa_indexer_score_topk_compressed(*a[:12], int(compress_ratio), *a[12:]))


def _score_args(q_fp8, q_scale, w, k_cache, query_start_loc, seq_lens, block_table, index_topk,
                topk_buffer, workspace, scores_out, status, stream):
    T, H = q_fp8.shape[0], q_fp8.shape[1]
    R = seq_lens.shape[0]
    _need(q_fp8, "q_fp8", torch.uint8, (T, H, HEAD_DIM))
    _need(q_scale, "q_scale", torch.float32, (T, H))
    _need(w, "w", torch.float32, (T, H))
    _need(k_cache, "k_cache", torch.uint8, (None, PAGE_BYTES))
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(topk_buffer, "topk_buffer", torch.int32, (None, index_topk))
    _need(workspace, "workspace", torch.uint8)
    ld = 0
    if scores_out is not None:
        _need(scores_out, "scores_out", torch.float32, (T, None))
        ld = scores_out.shape[1]
    if status is not None:
        _need(status, "status", torch.int32)
    return (_ptr(q_fp8), _ptr(q_scale), _ptr(w), T, H, _ptr(k_cache), k_cache.shape[0],
            _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table), block_table.shape[1],
            index_topk, _ptr(topk_buffer), topk_buffer.shape[0], _ptr(scores_out), ld,
            _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))


def score_topk_no_alloc(q_fp8: torch.Tensor, q_scale: torch.Tensor, w: torch.Tensor,
                        k_cache: torch.Tensor, query_start_loc: torch.Tensor,
                        seq_lens: torch.Tensor, block_table: torch.Tensor, index_topk: int,
                        topk_buffer: torch.Tensor, status: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """score_topk without a workspace argument: the library's built-in
    workspace is used and nothing is allocated (see include/dsa_indexer.h)."""
    T, H = q_fp8.shape[0], q_fp8.shape[1]
    R = seq_lens.shape[0]
    _need(q_fp8, "q_fp8", torch.uint8, (T, H, HEAD_DIM))
    _need(q_scale, "q_scale", torch.float32, (T, H))
    _need(w, "w", torch.float32, (T, H))
    _need(k_cache, "k_cache", torch.uint8, (None, PAGE_BYTES))
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(topk_buffer, "topk_buffer", torch.int32, (None, index_topk))
    if status is not None:
        _need(status, "status", torch.int32)
    _check(load().dsa_indexer_score_topk_no_alloc(
        _ptr(q_fp8), _ptr(q_scale), _ptr(w), T, H, _ptr(k_cache), k_cache.shape[0],
        _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table), block_table.shape[1],
        index_topk, _ptr(topk_buffer), topk_buffer.shape[0], _ptr(status), _stream(stream)))


def no_alloc_workspace_bytes() -> int:
    return int(load().dsa_indexer_no_alloc_workspace_bytes())


def layer_stack_run(layers: Sequence[Optional[dict]], pattern: Optional[str], freq: int,
                    offset: int, H: int, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                    block_table: torch.Tensor, num_pages: int, index_topk: int,
                    topk_buffer: torch.Tensor, workspace: torch.Tensor,
                    per_layer_out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                    slot_mapping: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, T: Optional[int] = None,
                    stream=None, compress_ratio: int = 1) -> None:
    """Run the F/S layer stack.  ``layers[l]`` is a dict with keys k, q_fp8,
    q_scale, w, k_cache (and optionally score_begin / score_end, torch.cuda.Event
    objects created with enable_timing=True) for F layers, or None for S layers.
    ``compress_ratio`` > 1 runs dsa_layer_stack_run_compressed (compressed
    caches, one entry per compress_ratio tokens)."""
    R = seq_lens.shape[0]
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(topk_buffer, "topk_buffer", torch.int32, (None, index_topk))
    _need(workspace, "workspace", torch.uint8)
    L = len(layers)
    arr = (LayerIO * L)()
    for i, io in enumerate(layers):
        if io is None:
            continue
        if T is None:
            T = io["k"].shape[0]
        _need(io["k"], f"layers[{i}].k", torch.float32, (T, HEAD_DIM))
        _need(io["q_fp8"], f"layers[{i}].q_fp8", torch.uint8, (T, H, HEAD_DIM))
        _need(io["q_scale"], f"layers[{i}].q_scale", torch.float32, (T, H))
        _need(io["w"], f"layers[{i}].w", torch.float32, (T, H))
        _need(io["k_cache"], f"layers[{i}].k_cache", torch.uint8, (num_pages, PAGE_BYTES))
        ev0, ev1 = io.get("score_begin"), io.get("score_end")
        arr[i] = LayerIO(io["k"].data_ptr(), io["q_fp8"].data_ptr(), io["q_scale"].data_ptr(),
                         io["w"].data_ptr(), io["k_cache"].data_ptr(),
                         None if ev0 is None else ev0.cuda_event,
                         None if ev1 is None else ev1.cuda_event)
    if T is None:
        raise ValueError("no F layer given")
    outs = None
    if per_layer_out is not None:
        outs = (ctypes.c_void_p * L)()
        for i, o in enumerate(per_layer_out):
            if o is not None:
                _need(o, f"per_layer_out[{i}]", torch.int32, (T, index_topk))
                outs[i] = o.data_ptr()
    if slot_mapping is not None:
        _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    if status is not None:
        _need(status, "status", torch.int32)
    head = (L, None if pattern is None else pattern.encode(), freq, offset, arr, T, H,
            _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table), block_table.shape[1],
            num_pages)
    tail = (index_topk, _ptr(topk_buffer), topk_buffer.shape[0], outs, _ptr(slot_mapping),
            _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    if compress_ratio == 1:
        _check(load().dsa_layer_stack_run(*head, *tail))
    else:
        _check(load().dsa_layer_stack_run_compressed(*head, int(compress_ratio), *tail))


def layer_stack_run_compressed(*args, compress_ratio: int, **kw) -> None:
    """dsa_layer_stack_run_compressed: layer_stack_run's arguments plus the ratio."""
    layer_stack_run(*args, compress_ratio=compress_ratio, **kw)


def layer_stack_run_bf16(layers: Sequence[Optional[dict]], pattern: Optional[str], freq: int,
                         offset: int, H: int, query_start_loc: torch.Tensor,
                         seq_lens: torch.Tensor, block_table: torch.Tensor, num_pages: int,
                         index_topk: int, topk_buffer: torch.Tensor, workspace: torch.Tensor,
                         per_layer_out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                         slot_mapping: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, T: Optional[int] = None,
                         stream=None) -> None:
    """The F/S layer stack with BF16 inputs.  ``layers[l]`` is a dict with keys
    k [T, 128] and q [T, H, 128] (BF16), w, k_cache, and the scratch q_fp8 /
    q_scale that the cache-write launch fills, for F layers; None for S
    layers."""
    R = seq_lens.shape[0]
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(topk_buffer, "topk_buffer", torch.int32, (None, index_topk))
    _need(workspace, "workspace", torch.uint8)
    L = len(layers)
    arr = (LayerIOBf16 * L)()
    for i, io in enumerate(layers):
        if io is None:
            continue
        if T is None:
            T = io["k"].shape[0]
        _need(io["k"], f"layers[{i}].k", torch.bfloat16, (T, HEAD_DIM))
        _need(io["q"], f"layers[{i}].q", torch.bfloat16, (T, H, HEAD_DIM))
        _need(io["w"], f"layers[{i}].w", torch.float32, (T, H))
        _need(io["k_cache"], f"layers[{i}].k_cache", torch.uint8, (num_pages, PAGE_BYTES))
        _need(io["q_fp8"], f"layers[{i}].q_fp8", torch.uint8, (T, H, HEAD_DIM))
        _need(io["q_scale"], f"layers[{i}].q_scale", torch.float32, (T, H))
        ev0, ev1 = io.get("score_begin"), io.get("score_end")
        arr[i] = LayerIOBf16(io["k"].data_ptr(), io["q"].data_ptr(), io["w"].data_ptr(),
                             io["k_cache"].data_ptr(), io["q_fp8"].data_ptr(),
                             io["q_scale"].data_ptr(),
                             None if ev0 is None else ev0.cuda_event,
                             None if ev1 is None else ev1.cuda_event)
    if T is None:
        raise ValueError("no F layer given")
    outs = None
    if per_layer_out is not None:
        outs = (ctypes.c_void_p * L)()
        for i, o in enumerate(per_layer_out):
            if o is not None:
                _need(o, f"per_layer_out[{i}]", torch.int32, (T, index_topk))
                outs[i] = o.data_ptr()
    if slot_mapping is not None:
        _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    if status is not None:
        _need(status, "status", torch.int32)
    _check(load().dsa_layer_stack_run_bf16(
        L, None if pattern is None else pattern.encode(), freq, offset, arr, T, H,
        _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table), block_table.shape[1],
        num_pages, index_topk, _ptr(topk_buffer), topk_buffer.shape[0], outs, _ptr(slot_mapping),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))


# ---------------------------------------------------------------- sparse MLA
MLA_DIM = 576
MLA_LATENT = 512
MLA_RECORD_BYTES = 656
MLA_PAGE_BYTES = 41984


def mla_write_kv(kv: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                 block_table: torch.Tensor, kv_cache: torch.Tensor,
                 slot_mapping: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Store each new token's [latent | RoPE] (FP32 [T, 576]) as its 656-byte
    record in kv_cache [num_pages, 41984] (dsa_mla_write_kv)."""
    T = kv.shape[0]
    R = seq_lens.shape[0]
    _need(kv, "kv", torch.float32, (T, MLA_DIM))
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(kv_cache, "kv_cache", torch.uint8, (None, MLA_PAGE_BYTES))
    if slot_mapping is not None:
        _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    if status is not None:
        _need(status, "status", torch.int32)
    _check(load().dsa_mla_write_kv(
        _ptr(kv), T, _ptr(query_start_loc), _ptr(seq_lens), R, _ptr(block_table),
        block_table.shape[1], _ptr(kv_cache), kv_cache.shape[0], _ptr(slot_mapping),
        _ptr(status), _stream(stream)))


def sparse_mla_attention(q: torch.Tensor, kv_cache: torch.Tensor, query_start_loc: torch.Tensor,
                         seq_lens: torch.Tensor, block_table: torch.Tensor,
                         topk_indices: torch.Tensor, softmax_scale: float,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None):
    """Attention of each query row (q [T, Hq, 576] BF16) over the tokens its
    top-k row selects (dsa_sparse_mla_attention).  Returns (out [T, Hq, 512]
    BF16, lse [T, Hq] FP32)."""
    T, Hq = q.shape[0], q.shape[1]
    R = seq_lens.shape[0]
    _need(q, "q", torch.bfloat16, (T, Hq, MLA_DIM))
    _need(kv_cache, "kv_cache", torch.uint8, (None, MLA_PAGE_BYTES))
    _need(query_start_loc, "query_start_loc", torch.int32, (R + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (R,))
    _need(block_table, "block_table", torch.int32, (R, None))
    _need(topk_indices, "topk_indices", torch.int32, (None, None))
    if topk_indices.shape[0] < T:
        raise ValueError("topk_indices has fewer rows than q")
    if out is None:
        out = _empty((T, Hq, MLA_LATENT), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, stream)
    _need(out, "out", torch.bfloat16, (T, Hq, MLA_LATENT))
    _need(lse, "lse", torch.float32, (T, Hq))
    if status is not None:
        _need(status, "status", torch.int32)
    _check(load().dsa_sparse_mla_attention(
        _ptr(q), T, Hq, _ptr(kv_cache), kv_cache.shape[0], _ptr(query_start_loc),
        _ptr(seq_lens), R, _ptr(block_table), block_table.shape[1], _ptr(topk_indices),
        topk_indices.shape[1], float(softmax_scale), _ptr(out), _ptr(lse), _ptr(status),
        _stream(stream)))
    return out, lse


# ------------------------------------------- tables, K/V cache, attention, norm
# These calls are made for every layer and step, some with a few microseconds of
# GPU work: their checks take the short way where everything is as it should be.
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
TYPE_E4M3 = 3
NORM_GROUP = 128
_KV_CACHE = struct.Struct("@4P11q3i")   # KvCache's fields
_raw_stream = torch._C._cuda_getCurrentRawStream
_Tensor = torch.Tensor


def _stream_of(stream, device: int) -> int:
    """The stream to launch on: the device's current one unless given."""
    if stream is None:
        return _raw_stream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is one of cuda:{stream.device_index}, the tensors lie on cuda:{device}")
    return stream.cuda_stream


def _device_of(t: torch.Tensor, name: str) -> int:
    """The device of a call's tensors, which has to be the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device != _current_device():
        _refuse_device(device, name)
    return device


def _full(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> int:
    """The address of a contiguous tensor of this dtype and shape on `device`, the current one."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == device and t.is_contiguous()):
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} is not as it should be: {dtype} {shape} on cuda:{device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> tuple:
    """The strides of a tensor of this dtype and shape on `device` whose last
    dimension is contiguous."""
    strides = t.stride()
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and (strides[-1] == 1 or shape[-1] == 1)):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        _device_of(t, name)
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return strides


def _type_of(t: torch.Tensor, name: str, most: int = 1) -> int:
    kind = TYPES.get(t.dtype)
    if kind is None or kind > most:
        wanted = ", ".join(str(d) for d, k in TYPES.items() if k <= most)
        raise TypeError(f"{name} must be one of {wanted}, got {t.dtype}")
    return kind


def _status(status: Optional[torch.Tensor], device: int) -> Optional[int]:
    if status is None:
        return None
    _need(status, "status", torch.int32)
    return status.data_ptr()


def build_block_tables(query_lens: torch.Tensor, seq_lens: torch.Tensor, free_pages: torch.Tensor,
                       block_table: torch.Tensor, query_start_loc: torch.Tensor,
                       positions: torch.Tensor, slot_mapping: torch.Tensor,
                       pages_used: torch.Tensor, status: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """A step's block tables and slot maps from the requests' lengths
    (dsa_block_tables_build): block_table [R, max_blocks] gains the new pages
    (taken from free_pages in request order), and query_start_loc [R+1],
    positions [T], slot_mapping [T] and pages_used [1] are written."""
    dev = _device_of(query_lens, "query_lens")
    R, T = query_lens.shape[0], positions.shape[0]
    num_free, max_blocks = free_pages.shape[0], block_table.shape[-1]
    i32 = torch.int32
    rc = load().dsa_block_tables_build(
        _full(query_lens, "query_lens", i32, (R,), dev), _full(seq_lens, "seq_lens", i32, (R,), dev), R,
        _full(free_pages, "free_pages", i32, (num_free,), dev), num_free,
        _full(block_table, "block_table", i32, (R, max_blocks), dev), max_blocks, T,
        _full(query_start_loc, "query_start_loc", i32, (R + 1,), dev),
        _full(positions, "positions", i32, (T,), dev),
        _full(slot_mapping, "slot_mapping", torch.int64, (T,), dev),
        _full(pages_used, "pages_used", i32, (1,), dev), _status(status, dev), _stream_of(stream, dev))
    if rc:
        _check(rc)


def _kv_cache(k_cache, v_cache, k_scale, v_scale, like, heads, dim, device) -> bytes:
    """The C description (KvCache) of a paged K/V cache after checking its tensors."""
    pages, dtype = k_cache.shape[0], k_cache.dtype
    if dtype is torch.uint8:
        if k_scale is None or v_scale is None:
            raise ValueError("a uint8 (E4M3) cache needs k_scale and v_scale")
        kind, shape = TYPE_E4M3, (pages, heads, PAGE_TOKENS)
        sk = _rows(k_scale, "k_scale", torch.float32, shape, device)
        sv = _rows(v_scale, "v_scale", torch.float32, shape, device)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    else:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales go with a uint8 (E4M3) cache")
        if dtype is not like.dtype:
            raise TypeError(f"k_cache must be {like.dtype} or torch.uint8, got {dtype}")
        kind, sk, sv, ks, vs = TYPES[dtype], (0, 0), (0, 0), 0, 0
    shape = (pages, PAGE_TOKENS, heads, dim)
    a = _rows(k_cache, "k_cache", dtype, shape, device)
    b = _rows(v_cache, "v_cache", dtype, shape, device)
    return _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, a[0], a[1], a[2], b[0],
                          b[1], b[2], sk[0], sk[1], sv[0], sv[1], pages, heads, dim, kind)


def kv_write(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
             v_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
             stream=None) -> None:
    """Store the new tokens' keys and values (k, v [T, Hkv, D], BF16 or FP16)
    at their slots of k_cache, v_cache [num_pages, 64, Hkv, D] (dsa_kv_write):
    copied into caches of the same type, or quantised into uint8 (E4M3) caches
    with scales [num_pages, Hkv, 64]."""
    kind = _type_of(k, "k")
    dev = _device_of(k, "k")
    T, heads, dim = shape = tuple(k.shape)
    a = _rows(k, "k", k.dtype, shape, dev)
    b = _rows(v, "v", k.dtype, shape, dev)
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, k, heads, dim, dev)
    rc = load().dsa_kv_write(
        k.data_ptr(), a[0], a[1], v.data_ptr(), b[0], b[1], kind, T,
        _full(slot_mapping, "slot_mapping", torch.int64, (T,), dev), cache, _status(status, dev),
        _stream_of(stream, dev))
    if rc:
        _check(rc)


def attention_workspace_bytes() -> int:
    return int(load().dsa_paged_attention_workspace_bytes())


def alloc_attention_workspace(device="cuda") -> torch.Tensor:
    """A zeroed workspace for paged_attention, whatever the batch."""
    return torch.zeros(attention_workspace_bytes(), dtype=torch.uint8, device=device)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                    block_table: torch.Tensor, softmax_scale: float, workspace: torch.Tensor,
                    window: int = 0, num_sinks: int = 0, k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream=None):
    """Attention of the step's query rows (q [T, Hq, D], BF16 or FP16) over the
    paged K/V cache [num_pages, 64, Hkv, D], causal; window > 0 keeps the last
    `window` tokens and the first `num_sinks` (dsa_paged_attention).  Returns
    (out [T, Hq, D] like q, lse [T, Hq] FP32); where they are not given, their
    memory belongs to the stream of the launch."""
    kind = _type_of(q, "q")
    dev = _device_of(q, "q")
    T, Hq, dim = shape = tuple(q.shape)
    a = _rows(q, "q", q.dtype, shape, dev)
    cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, q, k_cache.shape[2], dim, dev)
    if out is None:
        out = _empty(shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, stream)
    b = _rows(out, "out", q.dtype, shape, dev)
    R, max_blocks, n_ws = seq_lens.shape[0], block_table.shape[-1], workspace.shape[0]
    i32 = torch.int32
    rc = load().dsa_paged_attention(
        q.data_ptr(), a[0], a[1], kind, T, Hq, cache,
        _full(query_start_loc, "query_start_loc", i32, (R + 1,), dev),
        _full(seq_lens, "seq_lens", i32, (R,), dev), R,
        _full(block_table, "block_table", i32, (R, max_blocks), dev), max_blocks, softmax_scale,
        window, num_sinks, out.data_ptr(), b[0], b[1], _full(lse, "lse", torch.float32, (T, Hq), dev),
        _full(workspace, "workspace", torch.uint8, (n_ws,), dev), n_ws, _status(status, dev),
        _stream_of(stream, dev))
    if rc:
        _check(rc)
    return out, lse


def add_rms_norm(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor,
                 eps: float, residual_out: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """h = x + residual (rounded to x's type, written to residual_out) and its
    root-mean-square norm y (dsa_add_rms_norm): rounded to `out`, and / or
    quantised to codes [T, N] uint8 (E4M3) with scales [T, ceil(N/128)].  x,
    residual, residual_out, out [T, N] may have any row stride; residual_out
    may be x or residual."""
    kind = _type_of(x, "x", most=2)
    dev, dtype = _device_of(x, "x"), x.dtype
    T, N = shape = tuple(x.shape)

    def row(t, name):  # address and row stride
        if t is None:
            return None, N
        strides = _rows(t, name, dtype, shape, dev)
        return t.data_ptr(), strides[0] if T > 1 else N

    args = [*row(x, "x"), *row(residual, "residual")]
    args += [_full(weight, "weight", dtype, (N,), dev), kind, T, N, eps]
    args += [*row(residual_out, "residual_out"), *row(out, "out")]
    args.append(None if codes is None else _full(codes, "codes", torch.uint8, (T, N), dev))
    args.append(None if scales is None else
                _full(scales, "scales", torch.float32, (T, -(-N // NORM_GROUP)), dev))
    rc = load().dsa_add_rms_norm(*args, _stream_of(stream, dev))
    if rc:
        _check(rc)


# ------------------------------------------- products, router, weighted sum
SCORINGS = {"sigmoid": 0, "softmax": 1}


def _matmul_out(M, N, gated, x, dtype, out, out_codes, out_scales, device, stream):
    """The outputs of a product, checked: what it returns, and the entry point's arguments for them."""
    if gated:
        if N % 2:
            raise ValueError(f"gated weights have two halves: {N} rows are odd")
        N //= 2
    if out_codes is not None or out_scales is not None:
        if out is not None:
            raise ValueError("either out or out_codes and out_scales")
        if out_codes is None or out_scales is None:
            raise ValueError("out_codes and out_scales are given together")
        return (out_codes, out_scales), (
            None, N, 0, _full(out_codes, "out_codes", torch.uint8, (M, N), device),
            _full(out_scales, "out_scales", torch.float32, (M, (N + 127) // 128), device))
    if out is None:
        out = _empty((M, N), dtype, x.device, stream)
    kind = _type_of(out, "out", most=2)
    strides = _rows(out, "out", out.dtype, (M, N), device)
    return out, (out.data_ptr(), strides[0] if M > 1 else N, kind, None, None)


def fp8_matmul(codes: torch.Tensor, scales: torch.Tensor, w_codes: torch.Tensor,
               w_scales: torch.Tensor, gated: bool = False, out: Optional[torch.Tensor] = None,
               out_codes: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None,
               stream=None):
    """Product of 8-bit rows (codes [T, K] uint8 E4M3, scales [T, ceil(K/128)], as add_rms_norm
    writes them) and weights (w_codes [N, K], w_scales [ceil(N/128), ceil(K/128)])
    (dsa_fp8_matmul).  gated: silu of the first half times the second, N/2 wide; with out_codes
    [T, N/2] uint8 and out_scales [T, ceil(N/256)] the result is quantised for the next product.
    Returns out [T, N or N/2] (allocated as out_dtype, of the stream of the launch, where it is
    not given), or (out_codes, out_scales)."""
    dev = _device_of(codes, "codes")
    T, K = shape = codes.shape
    N, kb = w_codes.shape[0], (K + 127) // 128
    f32, u8 = torch.float32, torch.uint8
    a = _rows(codes, "codes", u8, shape, dev)
    b = _rows(w_codes, "w_codes", u8, (N, K), dev)
    got, (o, o_stride, o_type, o_codes, o_scales) = _matmul_out(T, N, gated, codes, out_dtype, out, out_codes, out_scales, dev, stream)
    rc = load().dsa_fp8_matmul(
        codes.data_ptr(), a[0], _full(scales, "scales", f32, (T, kb), dev), T, w_codes.data_ptr(), b[0],
        _full(w_scales, "w_scales", f32, ((N + 127) // 128, kb), dev), N, K, gated, o, o_stride, o_type,
        o_codes, o_scales, None if status is None else _status(status, dev), _stream_of(stream, dev))
    if rc:
        _check(rc)
    return got


def grouped_matmul(x: torch.Tensor, weight: torch.Tensor, group_starts: torch.Tensor,
                   x_scales: Optional[torch.Tensor] = None,
                   w_scales: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                   gated: bool = False, out: Optional[torch.Tensor] = None,
                   out_codes: Optional[torch.Tensor] = None,
                   out_scales: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, status: Optional[torch.Tensor] = None,
                   stream=None):
    """Products grouped by expert (dsa_grouped_matmul): rows group_starts[e] to group_starts[e+1]
    times weight[e] of weight [E, N, K].  Row i is x[rows[i]] (rows [M] int32, as route_experts
    makes them), or x[i] without rows.  x [S, K] and weight are uint8 (E4M3) with x_scales [S,
    ceil(K/128)] and w_scales [E, ceil(N/128), ceil(K/128)], or both BF16 or FP16.  gated, the
    outputs [M, ..] and what is returned: as fp8_matmul; out_dtype is x's own unless given (BF16
    of 8-bit rows).  Rows in no group are left as they were."""
    dev = _device_of(x, "x")
    S, K = shape = x.shape
    if weight.dim() != 3:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected (groups, rows, {K})")
    E, N = weight.shape[:2]
    own = x.dtype
    if own is torch.uint8:
        if x_scales is None or w_scales is None:
            raise ValueError("uint8 (E4M3) rows and weights need x_scales and w_scales")
        kind, kb, f32 = TYPE_E4M3, (K + 127) // 128, torch.float32
        xs = _full(x_scales, "x_scales", f32, (S, kb), dev)
        ws = _full(w_scales, "w_scales", f32, (E, (N + 127) // 128, kb), dev)
    else:
        kind, xs, ws = _type_of(x, "x"), None, None
        if x_scales is not None or w_scales is not None:
            raise ValueError("scales go with uint8 (E4M3) rows and weights")
    a = _rows(x, "x", own, shape, dev)
    b = _rows(weight, "weight", own, (E, N, K), dev)
    M, index = S, None
    if rows is not None:
        M = rows.shape[0]
        index = _full(rows, "rows", torch.int32, (M,), dev)
    got, (o, o_stride, o_type, o_codes, o_scales) = _matmul_out(
        M, N, gated, x, out_dtype or (torch.bfloat16 if kind == TYPE_E4M3 else own), out, out_codes, out_scales, dev, stream)
    rc = load().dsa_grouped_matmul(
        x.data_ptr(), a[0], xs, kind, S, index, M, weight.data_ptr(), b[1], b[0], ws, N, K,
        _full(group_starts, "group_starts", torch.int32, (E + 1,), dev), E, gated, o, o_stride, o_type,
        o_codes, o_scales, None if status is None else _status(status, dev), _stream_of(stream, dev))
    if rc:
        _check(rc)
    return got


def route_experts(logits: torch.Tensor, top_k: int, expert_ids: torch.Tensor,
                  weights: torch.Tensor, group_starts: torch.Tensor, rows: torch.Tensor,
                  places: torch.Tensor, scoring: str = "sigmoid",
                  bias: Optional[torch.Tensor] = None, num_groups: int = 1, top_groups: int = 1,
                  normalize: bool = True, scale: float = 1.0,
                  num_tokens: Optional[torch.Tensor] = None, stream=None) -> None:
    """Each token's top_k experts by logits [T, E] and the groups that they make
    (dsa_route_experts): expert_ids, weights (FP32) and places [T, top_k], group_starts [E+1]
    and rows [T * top_k] are written (int32).  scoring is "sigmoid" or "softmax"; bias [E] FP32
    counts in the choice alone; num_groups > 1 chooses within the best top_groups runs of
    experts; num_tokens [1] int32 (query_start_loc[-1:]) leaves padding rows out."""
    dev = _device_of(logits, "logits")
    kind = _type_of(logits, "logits", most=2)
    T, E = shape = logits.shape
    if scoring not in SCORINGS:
        raise ValueError(f"scoring must be one of {', '.join(SCORINGS)}, got {scoring!r}")
    a = _rows(logits, "logits", logits.dtype, shape, dev)
    i32, pairs = torch.int32, (T, top_k)
    rc = load().dsa_route_experts(
        logits.data_ptr(), a[0] if T > 1 else E, kind,
        None if bias is None else _full(bias, "bias", torch.float32, (E,), dev), T, E, top_k,
        SCORINGS[scoring], num_groups, top_groups, normalize, scale,
        None if num_tokens is None else _full(num_tokens, "num_tokens", i32, (1,), dev),
        _full(expert_ids, "expert_ids", i32, pairs, dev), _full(weights, "weights", torch.float32, pairs, dev),
        _full(group_starts, "group_starts", i32, (E + 1,), dev), _full(rows, "rows", i32, (T * top_k,), dev),
        _full(places, "places", i32, pairs, dev), _stream_of(stream, dev))
    if rc:
        _check(rc)


def combine_experts(y: torch.Tensor, places: torch.Tensor, weights: torch.Tensor,
                    add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * y[places[t, j]] (dsa_combine_experts): the experts'
    rows y [M, N] back to their tokens, places and weights [T, top_k] as route_experts writes
    them.  add and out [T, N] of y's type with any row stride; add may be out.  Returns out."""
    dev = _device_of(y, "y")
    kind, dtype = _type_of(y, "y", most=2), y.dtype
    M, N = shape = y.shape
    T, top_k = pairs = places.shape
    a = _rows(y, "y", dtype, shape, dev)
    if out is None:
        out = _empty((T, N), dtype, y.device, stream)
    b = _rows(out, "out", dtype, (T, N), dev)
    c = b if add is None else _rows(add, "add", dtype, (T, N), dev)
    rc = load().dsa_combine_experts(
        y.data_ptr(), a[0] if M > 1 else N, kind, M, _full(places, "places", torch.int32, pairs, dev),
        _full(weights, "weights", torch.float32, pairs, dev), T, top_k, N,
        None if add is None else add.data_ptr(), c[0] if T > 1 else N, out.data_ptr(), b[0] if T > 1 else N,
        None if status is None else _status(status, dev), _stream_of(stream, dev))
    if rc:
        _check(rc)
    return out

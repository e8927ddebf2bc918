"""Python binding of libpagedattn.so (include/pagedattn.h), via ctypes.

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of the library.  Tensors are torch CUDA tensors; their data pointers
and torch's current CUDA stream are handed to the C ABI unchanged.  If the
library has not been built, importing works but every call raises -- there is
no CPU fallback.

Names follow the C ABI: paged_kv_append, paged_attention_decode,
paged_attention_decode_append (both in one launch), paged_kv_append_tokens
(prefill write), paged_attention_decode_window (sliding window),
paged_attention_partial_workspace, paged_attention_decode_partial,
paged_attention_decode_reduce, paged_attention_decode_path,
paged_attention_decode_kernel (which kernel runs a shape on this device),
paged_attention_balanced_workspace, paged_attention_decode_balanced
(persistent load-balanced schedule), paged_kv_append_int8,
paged_attention_decode_int8 (int8 cache with per-block scales),
paged_kv_append_fp8, paged_attention_decode_fp8 (fp8 E4M3 cache with
per-block scales), paged_kv_append_rope (per-head norm, position rotation and
append in one pass; include/pagedattn_rope.h), paged_kv_append_fp4,
paged_kv_append_rope_fp4, paged_attention_decode_fp4, paged_kv_gather_fp4 (the
4-bit cache; include/pagedattn_fp4.h), paged_kv_append_rope_axes (positions of
several axes; include/pagedattn_axes.h), paged_attention_chunk,
paged_attention_chunk_diff (attention of several new tokens per sequence, and
its differential form; include/pagedattn_chunk.h).
"""
from __future__ import annotations

import ctypes
import struct
import threading
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "_lib" / "libpagedattn.so"

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_MISALIGNED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(6)
PA_F32, PA_F16, PA_BF16 = 0, 1, 2
PA_PATH_INVALID, PA_PATH_SIMT, PA_PATH_TENSOR_GQA = 0, 1, 2
PA_KERNEL_INVALID, PA_KERNEL_SIMT, PA_KERNEL_MMA_SYNC, PA_KERNEL_TCGEN05 = 0, 1, 2, 3
DEVERR_BAD_LEN, DEVERR_BAD_BLOCK, DEVERR_BAD_POS, DEVERR_TIMEOUT, DEVERR_BAD_PREFIX = 1, 2, 4, 8, 16

EXPORTED = ("pa_status_string", "pa_version", "paged_kv_append", "paged_attention_decode",
            "paged_attention_decode_append", "paged_attention_decode_split_static",
            "paged_kv_append_tokens", "paged_attention_decode_window",
            "paged_attention_decode_path", "paged_attention_decode_kernel",
            "paged_attention_partial_workspace",
            "paged_attention_decode_partial", "paged_attention_decode_reduce",
            "paged_attention_balanced_workspace", "paged_attention_decode_balanced",
            "paged_kv_append_int8", "paged_attention_decode_int8",
            "paged_kv_append_fp8", "paged_attention_decode_fp8",
            "paged_attention_decode_shared_prefix", "paged_attention_decode_shared_prefix_int8",
            "paged_attention_decode_shared_prefix_fp8",
            "paged_kv_append_rope", "paged_kv_append_fp4", "paged_kv_append_rope_fp4",
            "paged_kv_gather_fp4", "paged_attention_fp4_workspace", "paged_attention_decode_fp4",
            "paged_kv_append_rope_axes", "paged_attention_chunk_workspace", "paged_attention_chunk",
            "paged_attention_chunk_diff")


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class Shape(ctypes.Structure):
    """Mirror of pa_shape."""
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64), ("block_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class Rope(ctypes.Structure):
    """Mirror of pa_rope."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_position", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


class NewRows(ctypes.Structure):
    """Mirror of pa_new_rows."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("max_tokens", ctypes.c_int32)]


class RopeAxes(ctypes.Structure):
    """Mirror of pa_rope_axes."""
    _fields_ = [("positions", ctypes.c_void_p), ("num_axes", ctypes.c_int32), ("pair_axis", ctypes.c_void_p)]


class Diff(ctypes.Structure):
    """Mirror of pa_diff."""
    _fields_ = [("lambdas", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("out_scale", ctypes.c_float)]


# The structs as bytes (a third of a Structure's time to build).
_SHAPE, _ROPE, _ROWS = struct.Struct("@6i2qi0q"), struct.Struct("@P3i2Pf0q"), struct.Struct("@3P3qi0q")
_DIFF, _AXES = struct.Struct("@2P2f0q"), struct.Struct("@PiP")
assert [s.size for s in (_SHAPE, _ROPE, _ROWS, _DIFF, _AXES)] == \
    [ctypes.sizeof(t) for t in (Shape, Rope, NewRows, Diff, RopeAxes)]

_lock = threading.Lock()
_lib = None


def load() -> ctypes.CDLL:
    """Load the in-tree library; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not LIB_PATH.exists():
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(str(LIB_PATH))
            vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
            sp = ctypes.POINTER(Shape)
            lib.pa_status_string.restype = ctypes.c_char_p
            lib.pa_status_string.argtypes = [ctypes.c_int]
            lib.pa_version.restype = i32
            lib.pa_version.argtypes = []
            lib.paged_kv_append.restype = ctypes.c_int
            lib.paged_kv_append.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.paged_attention_decode.restype = ctypes.c_int
            lib.paged_attention_decode.argtypes = [sp, vp, vp, vp, vp, vp, vp, f32, vp, vp]
            lib.paged_attention_decode_append.restype = ctypes.c_int
            lib.paged_attention_decode_append.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, f32,
                                                          vp, vp]
            lib.paged_kv_append_tokens.restype = ctypes.c_int
            lib.paged_kv_append_tokens.argtypes = [sp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp]
            lib.paged_attention_decode_window.restype = ctypes.c_int
            lib.paged_attention_decode_window.argtypes = [sp, vp, vp, vp, vp, vp, vp, f32, i32, vp,
                                                          vp]
            lib.paged_attention_decode_path.restype = ctypes.c_int
            lib.paged_attention_decode_path.argtypes = [sp]
            lib.paged_attention_decode_kernel.restype = ctypes.c_int
            lib.paged_attention_decode_kernel.argtypes = [sp, i32, i32]
            lib.paged_attention_partial_workspace.restype = sz
            lib.paged_attention_partial_workspace.argtypes = [sp, i32]
            lib.paged_attention_decode_partial.restype = ctypes.c_int
            lib.paged_attention_decode_partial.argtypes = [sp, vp, vp, vp, vp, vp, f32, i32, vp, sz,
                                                           vp, vp]
            lib.paged_attention_decode_reduce.restype = ctypes.c_int
            lib.paged_attention_decode_reduce.argtypes = [sp, vp, vp, sz, vp, i32, vp, vp]
            lib.paged_attention_decode_shared_prefix.restype = ctypes.c_int
            lib.paged_attention_decode_shared_prefix.argtypes = [sp, vp, vp, vp, vp, vp, vp, i32, vp, vp,
                                                                 f32, i32, vp, sz, vp, vp]
            for name in ("paged_attention_decode_shared_prefix_int8", "paged_attention_decode_shared_prefix_fp8"):
                fn = getattr(lib, name)
                fn.restype = ctypes.c_int
                fn.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, f32, i32, vp, sz, vp, vp]
            lib.paged_kv_append_int8.restype = ctypes.c_int
            lib.paged_kv_append_int8.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.paged_attention_decode_int8.restype = ctypes.c_int
            lib.paged_attention_decode_int8.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp]
            lib.paged_kv_append_fp8.restype = ctypes.c_int
            lib.paged_kv_append_fp8.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.paged_attention_decode_fp8.restype = ctypes.c_int
            lib.paged_attention_decode_fp8.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp]
            lib.paged_attention_balanced_workspace.restype = sz
            lib.paged_attention_balanced_workspace.argtypes = [sp]
            lib.paged_attention_decode_balanced.restype = ctypes.c_int
            lib.paged_attention_decode_balanced.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                            f32, i32, vp, sz, vp, vp]
            # structs by address: a Structure's byref, or its bytes
            lib.paged_kv_append_rope.restype = ctypes.c_int
            lib.paged_kv_append_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.paged_kv_append_fp4.restype = ctypes.c_int
            lib.paged_kv_append_fp4.argtypes = [vp, vp, vp, vp, vp, f32, f32, vp, vp, vp, vp, vp]
            lib.paged_kv_append_rope_fp4.restype = ctypes.c_int
            lib.paged_kv_append_rope_fp4.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, f32, vp, vp, vp, vp, vp]
            lib.paged_kv_gather_fp4.restype = ctypes.c_int
            lib.paged_kv_gather_fp4.argtypes = [vp, vp, vp, i32, vp, vp, vp, f32, f32, vp, vp, vp, vp, vp]
            lib.paged_attention_fp4_workspace.restype = sz
            lib.paged_attention_fp4_workspace.argtypes = [sp]
            lib.paged_attention_decode_fp4.restype = ctypes.c_int
            lib.paged_attention_decode_fp4.argtypes = [vp, vp, vp, vp, vp, vp, f32, f32, vp, vp, f32, i32, vp, sz,
                                                       vp, vp]
            lib.paged_kv_append_rope_axes.restype = ctypes.c_int
            lib.paged_kv_append_rope_axes.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.paged_attention_chunk_workspace.restype = sz
            lib.paged_attention_chunk_workspace.argtypes = [sp]
            lib.paged_attention_chunk.restype = ctypes.c_int
            lib.paged_attention_chunk.argtypes = [vp, vp, vp, ctypes.c_int64, i32, vp, vp, vp, vp, vp, f32, i32, vp, sz,
                                                  vp, vp]
            lib.paged_attention_chunk_diff.restype = ctypes.c_int
            lib.paged_attention_chunk_diff.argtypes = [vp, vp, vp, vp, ctypes.c_int64, i32, vp, vp, vp, vp, vp, f32, i32,
                                                       vp, sz, vp, vp]
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def version() -> int:
    return int(load().pa_version())


_DTYPE_CODES = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}


def dtype_code(dtype: torch.dtype) -> int:
    try:
        return _DTYPE_CODES[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None


def make_shape(*, batch, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
               num_blocks, block_stride, dtype) -> Shape:
    return Shape(int(batch), int(num_heads), int(num_kv_heads), int(head_dim), int(block_size),
                 int(max_blocks_per_seq), int(num_blocks), int(block_stride),
                 dtype if isinstance(dtype, int) else dtype_code(dtype))


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status: int, what: str) -> None:
    if status != PA_OK:
        raise PagedAttnError(status, what)


class Prepared:
    """A C-ABI call with its arguments marshalled once.

    Calling it re-issues the same call (same buffers, shape, scale and
    stream), costing a few microseconds of host time instead of the full
    marshalling; the tensors it was built from must stay alive and keep their
    storage.  Every wrapper below returns one when given prepare=True.
    """

    __slots__ = ("_fn", "_args", "_what", "_keep")

    def __init__(self, fn, args, what, keep):
        self._fn, self._args, self._what, self._keep = fn, args, what, keep

    def __call__(self) -> None:
        status = self._fn(*self._args)
        if status != PA_OK:
            raise PagedAttnError(status, self._what)


def _issue(fn, args, what, prepare, keep=()):
    if prepare:
        return Prepared(fn, args, what, keep)
    _check(fn(*args), what)
    return None


def decode_shape(q, block_table, *, num_kv_heads, block_size, num_blocks, block_stride) -> Shape:
    B, H, D = q.shape
    return make_shape(batch=B, num_heads=H, num_kv_heads=num_kv_heads, head_dim=D,
                      block_size=block_size, max_blocks_per_seq=block_table.shape[1],
                      num_blocks=num_blocks, block_stride=block_stride, dtype=q.dtype)


def paged_kv_append(k_new, v_new, k_pool, v_pool, block_table, positions, *, block_size,
                    num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    """Write k_new/v_new [B][Hkv][D] at positions[b] through block_table."""
    B, Hkv, D = k_new.shape
    shape = make_shape(batch=B, num_heads=Hkv, num_kv_heads=Hkv, head_dim=D, block_size=block_size,
                       max_blocks_per_seq=block_table.shape[1], num_blocks=num_blocks,
                       block_stride=block_stride, dtype=k_new.dtype)
    args = (
            ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool),
            _ptr(block_table), _ptr(positions), _ptr(err_word), _stream(stream))
    return _issue(load().paged_kv_append, args, "paged_kv_append", prepare,
                  (shape,))


def paged_attention_decode(out, q, k_pool, v_pool, block_table, seq_lens, scale, *, num_kv_heads,
                           block_size, num_blocks, block_stride, err_word=None,
                           stream=None, prepare=False):
    """out[B][H][D] = attention of q over the valid tokens of each sequence."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    args = (
            ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool),
            _ptr(block_table), _ptr(seq_lens), float(scale), _ptr(err_word), _stream(stream))
    return _issue(load().paged_attention_decode, args, "paged_attention_decode", prepare,
                  (shape,))


def paged_attention_decode_append(out, q, k_new, v_new, k_pool, v_pool, block_table, positions,
                                  scale, *, num_kv_heads, block_size, num_blocks, block_stride,
                                  err_word=None, stream=None, prepare=False):
    """Append k_new/v_new at positions[b], then attend over positions[b] + 1 tokens."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    args = (
            ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pool),
            _ptr(v_pool), _ptr(block_table), _ptr(positions), float(scale), _ptr(err_word),
            _stream(stream))
    return _issue(load().paged_attention_decode_append, args, "paged_attention_decode_append", prepare,
                  (shape,))


def paged_kv_append_tokens(k_new, v_new, k_pool, v_pool, block_table, positions, counts, *,
                           block_size, num_blocks, block_stride, err_word=None,
                           stream=None, prepare=False):
    """Prefill write: counts[b] rows of the padded batch k_new/v_new [B][T][Hkv][D]
    go to positions[b] + t."""
    B, T, Hkv, D = k_new.shape
    shape = make_shape(batch=B, num_heads=Hkv, num_kv_heads=Hkv, head_dim=D, block_size=block_size,
                       max_blocks_per_seq=block_table.shape[1], num_blocks=num_blocks,
                       block_stride=block_stride, dtype=k_new.dtype)
    args = (
            ctypes.byref(shape), _ptr(k_new), _ptr(v_new), int(T), _ptr(k_pool), _ptr(v_pool),
            _ptr(block_table), _ptr(positions), _ptr(counts), _ptr(err_word), _stream(stream))
    return _issue(load().paged_kv_append_tokens, args, "paged_kv_append_tokens", prepare,
                  (shape,))


def paged_attention_decode_window(out, q, k_pool, v_pool, block_table, seq_lens, scale, window,
                                  *, num_kv_heads, block_size, num_blocks, block_stride,
                                  err_word=None, stream=None, prepare=False):
    """Decode attention over the last `window` valid tokens of each sequence."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    args = (
            ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool),
            _ptr(block_table), _ptr(seq_lens), float(scale), int(window), _ptr(err_word),
            _stream(stream))
    return _issue(load().paged_attention_decode_window, args, "paged_attention_decode_window", prepare,
                  (shape,))


def paged_attention_decode_path(shape: Shape) -> int:
    return int(load().paged_attention_decode_path(ctypes.byref(shape)))


def paged_attention_decode_kernel(shape: Shape, window: int = 0, partition_tokens: int = 0) -> int:
    """PA_KERNEL_* the decode of `shape` runs on the current device (single
    pass, sliding window, or the split-KV partial pass when partition_tokens
    is positive)."""
    return load().paged_attention_decode_kernel(ctypes.byref(shape), window, partition_tokens)


def paged_attention_partial_workspace(shape: Shape, partition_tokens: int) -> int:
    return int(load().paged_attention_partial_workspace(ctypes.byref(shape), int(partition_tokens)))


def paged_attention_decode_partial(q, k_pool, v_pool, block_table, seq_lens, scale,
                                   partition_tokens, workspace, *, num_kv_heads, block_size,
                                   num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    nbytes = workspace.numel() * workspace.element_size()
    args = (
            ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
            _ptr(seq_lens), float(scale), int(partition_tokens), _ptr(workspace), nbytes,
            _ptr(err_word), _stream(stream))
    return _issue(load().paged_attention_decode_partial, args, "paged_attention_decode_partial", prepare,
                  (shape,))


def paged_attention_decode_reduce(out, workspace, seq_lens, partition_tokens, *, num_kv_heads,
                                  block_size, num_blocks, block_stride, max_blocks_per_seq,
                                  err_word=None, stream=None, prepare=False):
    B, H, D = out.shape
    shape = make_shape(batch=B, num_heads=H, num_kv_heads=num_kv_heads, head_dim=D,
                       block_size=block_size, max_blocks_per_seq=max_blocks_per_seq,
                       num_blocks=num_blocks, block_stride=block_stride, dtype=out.dtype)
    nbytes = workspace.numel() * workspace.element_size()
    args = (
            ctypes.byref(shape), _ptr(out), _ptr(workspace), nbytes, _ptr(seq_lens),
            int(partition_tokens), _ptr(err_word), _stream(stream))
    return _issue(load().paged_attention_decode_reduce, args, "paged_attention_decode_reduce", prepare,
                  (shape,))


def workspace_for(q, block_table, partition_tokens, *, num_kv_heads, block_size, num_blocks,
                  block_stride) -> torch.Tensor:
    """Allocate (through torch) a workspace big enough for the split-KV pair."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    n = paged_attention_partial_workspace(shape, partition_tokens)
    if n == 0:
        raise PagedAttnError(PA_ERR_INVALID_ARG, "paged_attention_partial_workspace")
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=q.device)


def paged_attention_balanced_workspace(shape: Shape) -> int:
    return int(load().paged_attention_balanced_workspace(ctypes.byref(shape)))


def balanced_workspace_for(q, block_table, *, num_kv_heads, block_size, num_blocks,
                           block_stride) -> torch.Tensor:
    """Allocate (through torch) a zero-filled workspace for
    paged_attention_decode_balanced on q's device."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    with torch.cuda.device(q.device):
        n = paged_attention_balanced_workspace(shape)
    if n == 0:
        raise PagedAttnError(PA_ERR_UNSUPPORTED, "paged_attention_balanced_workspace")
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=q.device)


def paged_attention_decode_balanced(out, q, k_pool, v_pool, block_table, scale, workspace, *,
                                    seq_lens=None, positions=None, k_new=None, v_new=None,
                                    window=0, num_kv_heads, block_size, num_blocks, block_stride,
                                    err_word=None, stream=None, prepare=False):
    """One decode step on the load-balanced persistent grid: plain decode
    (seq_lens) or fused append + decode (positions, k_new, v_new), over the
    last `window` tokens when window > 0."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    nbytes = workspace.numel() * workspace.element_size()
    args = (
            ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
            _ptr(seq_lens), _ptr(positions), _ptr(k_new), _ptr(v_new), float(scale), int(window),
            _ptr(workspace), nbytes, _ptr(err_word), _stream(stream))
    return _issue(load().paged_attention_decode_balanced, args, "paged_attention_decode_balanced",
                  prepare, (shape,))


def paged_kv_append_int8(k_new, v_new, k_pool, v_pool, kv_scales, block_table, positions, *,
                         block_size, num_blocks, block_stride, err_word=None, stream=None,
                         prepare=False):
    """Quantising append of k_new/v_new [B][Hkv][D] into int8 pools (codes of
    the target block's scales)."""
    B, Hkv, D = k_new.shape
    shape = make_shape(batch=B, num_heads=Hkv, num_kv_heads=Hkv, head_dim=D, block_size=block_size,
                       max_blocks_per_seq=block_table.shape[1], num_blocks=num_blocks,
                       block_stride=block_stride, dtype=k_new.dtype)
    args = (ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool),
            _ptr(kv_scales), _ptr(block_table), _ptr(positions), _ptr(err_word), _stream(stream))
    return _issue(load().paged_kv_append_int8, args, "paged_kv_append_int8", prepare, (shape,))


def paged_attention_decode_int8(out, q, k_pool, v_pool, kv_scales, block_table, seq_lens, scale, *,
                                num_kv_heads, block_size, num_blocks, block_stride, err_word=None,
                                stream=None, prepare=False):
    """Decode attention over an int8 cache with per-(block, kv head) scales."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    args = (ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(kv_scales),
            _ptr(block_table), _ptr(seq_lens), float(scale), _ptr(err_word), _stream(stream))
    return _issue(load().paged_attention_decode_int8, args, "paged_attention_decode_int8", prepare,
                  (shape,))


def paged_kv_append_fp8(k_new, v_new, k_pool, v_pool, kv_scales, block_table, positions, *,
                        block_size, num_blocks, block_stride, err_word=None, stream=None,
                        prepare=False):
    """Quantising append of k_new/v_new [B][Hkv][D] into fp8 (E4M3) pools
    (codes of the target block's scales)."""
    B, Hkv, D = k_new.shape
    shape = make_shape(batch=B, num_heads=Hkv, num_kv_heads=Hkv, head_dim=D, block_size=block_size,
                       max_blocks_per_seq=block_table.shape[1], num_blocks=num_blocks,
                       block_stride=block_stride, dtype=k_new.dtype)
    args = (ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool),
            _ptr(kv_scales), _ptr(block_table), _ptr(positions), _ptr(err_word), _stream(stream))
    return _issue(load().paged_kv_append_fp8, args, "paged_kv_append_fp8", prepare, (shape,))


def paged_attention_decode_fp8(out, q, k_pool, v_pool, kv_scales, block_table, seq_lens, scale, *,
                               num_kv_heads, block_size, num_blocks, block_stride, err_word=None,
                               stream=None, prepare=False):
    """Decode attention over an fp8 (E4M3) cache with per-(block, kv head)
    scales."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    args = (ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(kv_scales),
            _ptr(block_table), _ptr(seq_lens), float(scale), _ptr(err_word), _stream(stream))
    return _issue(load().paged_attention_decode_fp8, args, "paged_attention_decode_fp8", prepare,
                  (shape,))


def paged_attention_decode_shared_prefix(out, q, k_pool, v_pool, block_table, seq_lens, scale,
                                         partition_tokens, workspace, *, group_first, shared_tokens,
                                         num_kv_heads, block_size, num_blocks, block_stride,
                                         err_word=None, stream=None, prepare=False):
    """Split-KV decode where each group of sequences [group_first[i],
    group_first[i+1]) shares the blocks of its first shared_tokens[i] tokens:
    those partitions are read once per group (host lists)."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    n = len(shared_tokens)
    first = (ctypes.c_int32 * (n + 1))(*[int(x) for x in group_first])
    shared = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in shared_tokens])
    nbytes = workspace.numel() * workspace.element_size()
    args = (ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
            _ptr(seq_lens), n, ctypes.cast(first, ctypes.c_void_p), ctypes.cast(shared, ctypes.c_void_p),
            float(scale), int(partition_tokens), _ptr(workspace), nbytes, _ptr(err_word),
            _stream(stream))
    return _issue(load().paged_attention_decode_shared_prefix, args,
                  "paged_attention_decode_shared_prefix", prepare, (shape, first, shared))


def _shared_prefix_codes(name, out, q, k_pool, v_pool, kv_scales, block_table, seq_lens, scale,
                         partition_tokens, workspace, group_first, shared_tokens, num_kv_heads,
                         block_size, num_blocks, block_stride, err_word, stream, prepare):
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size,
                         num_blocks=num_blocks, block_stride=block_stride)
    n = len(shared_tokens)
    first = (ctypes.c_int32 * (n + 1))(*[int(x) for x in group_first])
    shared = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in shared_tokens])
    nbytes = workspace.numel() * workspace.element_size()
    args = (ctypes.byref(shape), _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(kv_scales),
            _ptr(block_table), _ptr(seq_lens), n, ctypes.cast(first, ctypes.c_void_p),
            ctypes.cast(shared, ctypes.c_void_p), float(scale), int(partition_tokens), _ptr(workspace),
            nbytes, _ptr(err_word), _stream(stream))
    return _issue(getattr(load(), name), args, name, prepare, (shape, first, shared))


def paged_attention_decode_shared_prefix_int8(out, q, k_pool, v_pool, kv_scales, block_table, seq_lens,
                                              scale, partition_tokens, workspace, *, group_first,
                                              shared_tokens, num_kv_heads, block_size, num_blocks,
                                              block_stride, err_word=None, stream=None, prepare=False):
    """paged_attention_decode_shared_prefix over an int8 cache with
    per-(block, kv head) scales (host group lists)."""
    return _shared_prefix_codes("paged_attention_decode_shared_prefix_int8", out, q, k_pool, v_pool,
                                kv_scales, block_table, seq_lens, scale, partition_tokens, workspace,
                                group_first, shared_tokens, num_kv_heads, block_size, num_blocks,
                                block_stride, err_word, stream, prepare)


def paged_attention_decode_shared_prefix_fp8(out, q, k_pool, v_pool, kv_scales, block_table, seq_lens,
                                             scale, partition_tokens, workspace, *, group_first,
                                             shared_tokens, num_kv_heads, block_size, num_blocks,
                                             block_stride, err_word=None, stream=None, prepare=False):
    """paged_attention_decode_shared_prefix over an fp8 (E4M3) cache with
    per-(block, kv head) scales (host group lists)."""
    return _shared_prefix_codes("paged_attention_decode_shared_prefix_fp8", out, q, k_pool, v_pool,
                                kv_scales, block_table, seq_lens, scale, partition_tokens, workspace,
                                group_first, shared_tokens, num_kv_heads, block_size, num_blocks,
                                block_stride, err_word, stream, prepare)


# ---------------------------------------------------------------------------
# norm, rotation and append in one pass; the 4-bit cache
# ---------------------------------------------------------------------------

def rope_table(max_position, rotary_dim, theta=10000.0, device=None) -> torch.Tensor:
    """cos_sin [max_position][rotary_dim] of the plain rotation: pair i turns by
    position * theta^(-2i/rotary_dim).  Angles in fp64, so far positions keep
    their precision; scaled rotations hand in a table of their own."""
    inv = float(theta) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    ang = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), 1).float()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # current_stream() without building a Stream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # of a process that has used one


def _launch_stream(stream, what, *tensors):
    """The stream a call runs on, after checking that every tensor (None aside)
    lies on the current device, the one the kernels are launched on."""
    dev = tensors[0].get_device()
    ok = dev >= 0 and dev == _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            ok = False
    if not ok:
        raise ValueError(f"{what}: all tensors must be on the current CUDA device")
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _dense(what, dtype, *tensors) -> None:
    for t in tensors:
        if t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous {dtype} tensors")


def _pools_hold(k_pool, v_pool, kv_scales, heads, D, block_size, num_blocks, block_stride) -> None:
    """Refuse pools and scales that end before num_blocks blocks do.  A pool is
    where its memory begins; how far it reaches, its storage says."""
    row = D if kv_scales is None else D // 2
    size = k_pool.element_size()
    need = ((num_blocks - 1) * block_stride + heads * block_size * row) * size
    for pool in (k_pool, v_pool):
        if pool.untyped_storage().nbytes() - pool.storage_offset() * size < need:
            raise ValueError("the pools must hold num_blocks blocks, block_stride apart")
    if kv_scales is not None and kv_scales.numel() < num_blocks * 2 * heads * block_size * (D // 16):
        raise ValueError("kv_scales must be [num_blocks][2][kv heads][block_size][head_dim/16]")


def _new_rows(what, x):
    """(batch, tokens, heads, head_dim, token stride) of new rows
    [B][heads][D] or [B][T][heads][D], possibly a slice of a packed
    projection output."""
    shape, strides = x.shape, x.stride()
    if len(shape) == 4:
        B, T, H, D = shape
        sb, stride, sh, sd = strides
        if T == 1:
            stride = sb
        elif B > 1 and T > 0 and sb != T * stride:
            raise ValueError(f"{what}: tokens must lie at one stride")
    elif len(shape) == 3:
        B, H, D = shape
        stride, sh, sd = strides
        T = 1
    else:
        raise ValueError(f"{what} must be [B][heads][D] or [B][T][heads][D]")
    if B * T <= 1:
        stride = H * D
    if (sd != 1 and D != 1) or (sh != D and H != 1):
        raise ValueError(f"{what}: the heads of a token must lie one after another")
    if stride < H * D:                         # expanded or overlapping tokens; 0 would mean rows without gaps
        raise ValueError(f"{what}: every token must have rows of its own")
    return B, T, H, D, stride


def _append_rows(name, q_out, q, k_new, v_new, k_pool, v_pool, kv_scales, k_scale, v_scale, block_table, positions,
                 counts, cos_sin, rotary_dim, interleaved, q_norm, k_norm, eps, block_size, num_blocks, block_stride,
                 err_word, stream, prepare, axis_positions=None, pair_axis=None):
    dt = k_new.dtype
    code = dtype_code(dt)
    B, T, Hkv, D, ks = _new_rows("k_new", k_new)
    b, t, h, d, vs = _new_rows("v_new", v_new)
    if b != B or t != T or h != Hkv or d != D or v_new.dtype != dt:
        raise ValueError("k_new and v_new differ in shape or dtype")
    H, qs, qp = Hkv, 0, 0
    if q is not None:
        b, t, H, d, qs = _new_rows("q", q)
        if b != B or t != T or d != D or q.dtype != dt:
            raise ValueError("q does not match the keys in batch, tokens, head_dim or dtype")
        if q_out is None or q_out.numel() != B * T * H * D or q_out.dtype != dt or not q_out.is_contiguous():
            raise ValueError(f"q_out must be contiguous, with batch * tokens * heads * head_dim elements of {dt}")
        qp = q.data_ptr()
    _dense("block_table and positions", torch.int32, block_table, positions)
    rows, MB = block_table.shape
    if rows != B or positions.numel() != B:
        raise ValueError("block_table and positions must have one row per sequence")
    if counts is not None and not (counts.dtype == torch.int32 and counts.is_contiguous() and counts.numel() == B):
        raise ValueError("counts must be a contiguous torch.int32 tensor with one entry per sequence")
    fp4 = kv_scales is not None
    if fp4:
        _dense("kv_scales", torch.uint8, kv_scales)
    pool_dtype = torch.uint8 if fp4 else dt
    if k_pool.dtype != pool_dtype or v_pool.dtype != pool_dtype:
        raise ValueError("the pools must be uint8 (4-bit cache) or of the new rows' dtype")
    _pools_hold(k_pool, v_pool, kv_scales, Hkv, D, block_size, num_blocks, block_stride)
    R, most = 0, 0
    if cos_sin is not None:
        _dense("cos_sin", torch.float32, cos_sin)
        most, R = cos_sin.shape
        if rotary_dim is not None and rotary_dim != R:
            raise ValueError("cos_sin must be [max_position][rotary_dim]")
    elif rotary_dim:
        raise ValueError("a rotation needs cos_sin")
    for w in (q_norm, k_norm):
        if w is not None and not (w.dtype == dt and w.is_contiguous() and w.numel() == D):
            raise ValueError(f"q_norm and k_norm must hold head_dim contiguous elements of {dt}")
    if pair_axis is not None:
        _dense("axis_positions", torch.int32, axis_positions)
        A = axis_positions.shape[0]
        if axis_positions.numel() != A * B * T or R == 0 or len(pair_axis) != R // 2:
            raise ValueError("axis_positions must be [axes][B][T], pair_axis rotary_dim/2 axes")
    on = _launch_stream(stream, name, k_new, v_new, q, q_out, k_pool, v_pool, kv_scales, block_table, positions, counts,
                        cos_sin, q_norm, k_norm, err_word, axis_positions)
    shape = _SHAPE.pack(B, H, Hkv, D, block_size, MB, num_blocks, block_stride, code)
    rows = _ROWS.pack(qp, k_new.data_ptr(), v_new.data_ptr(), qs, ks, vs, T)
    pools = (k_pool.data_ptr(), v_pool.data_ptr())
    if fp4:
        pools += (kv_scales.data_ptr(), k_scale, v_scale)
    tail = (block_table.data_ptr(), positions.data_ptr(), _addr(counts), _addr(err_word), on)
    if name == "paged_kv_append_fp4":
        return _issue(load().paged_kv_append_fp4, (shape, rows, *pools, *tail), name, prepare)
    rope = _ROPE.pack(_addr(cos_sin) or 0, most, R, interleaved, _addr(q_norm) or 0, _addr(k_norm) or 0, eps)
    if pair_axis is not None:
        pairs = ctypes.c_char_p(bytes(pair_axis))              # read before the call returns
        axes = _AXES.pack(axis_positions.data_ptr(), A, ctypes.cast(pairs, ctypes.c_void_p).value)
        return _issue(load().paged_kv_append_rope_axes, (shape, rope, axes, rows, _addr(q_out), *pools, *tail), name,
                      prepare, (pairs,))
    return _issue(getattr(load(), name), (shape, rope, rows, _addr(q_out), *pools, *tail), name, prepare)


def paged_kv_append_rope(q_out, q, k_new, v_new, k_pool, v_pool, block_table, positions, cos_sin, *,
                         counts=None, rotary_dim=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6,
                         block_size, num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    """Norm (q_norm, k_norm [D]) and rotate (cos_sin [max_position][rotary_dim],
    None: no rotation) the new queries and keys, write the queries to q_out and
    the keys and values at positions[b] + t through block_table.  q, k_new and
    v_new are [B][heads][D] or, with counts[b] valid tokens, [B][T][heads][D],
    slices of a packed projection output included; q may be None."""
    return _append_rows("paged_kv_append_rope", q_out, q, k_new, v_new, k_pool, v_pool, None, 1.0, 1.0, block_table,
                        positions, counts, cos_sin, rotary_dim, interleaved, q_norm, k_norm, eps, block_size,
                        num_blocks, block_stride, err_word, stream, prepare)


def rope_axes(sections, cyclic=False) -> bytes:
    """pair_axis of paged_kv_append_rope_axes: sections[a] pairs turn by axis a,
    one section after another or, cyclic, the axes in turn while they have
    pairs left."""
    left = [int(n) for n in sections]
    if min(left) < 0 or len(left) > 4:
        raise ValueError("rope_axes: up to 4 sections of 0 pairs or more")
    if not cyclic:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    return bytes(a for i in range(max(left)) for a, n in enumerate(left) if i < n)


def paged_kv_append_rope_axes(q_out, q, k_new, v_new, k_pool, v_pool, block_table, positions, axis_positions, cos_sin,
                              pair_axis, *, counts=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6,
                              block_size, num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    """paged_kv_append_rope for tokens with positions on several axes: pair i
    turns by axis_positions[pair_axis[i]] ([axes][B][T] int32); pair_axis is
    bytes (or ints) of rotary_dim/2 axes, see rope_axes."""
    if cos_sin is None or axis_positions is None or pair_axis is None or axis_positions.dim() == 0:
        raise ValueError("axes need cos_sin, axis_positions [axes][B][T] and pair_axis")
    return _append_rows("paged_kv_append_rope_axes", q_out, q, k_new, v_new, k_pool, v_pool, None, 1.0, 1.0, block_table,
                        positions, counts, cos_sin, None, interleaved, q_norm, k_norm, eps, block_size, num_blocks,
                        block_stride, err_word, stream, prepare, axis_positions, pair_axis)


def paged_kv_append_rope_fp4(q_out, q, k_new, v_new, k_pool, v_pool, kv_scales, block_table, positions, cos_sin, *,
                             counts=None, rotary_dim=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6,
                             k_scale=1.0, v_scale=1.0, block_size, num_blocks, block_stride, err_word=None,
                             stream=None, prepare=False):
    """paged_kv_append_rope into the 4-bit cache: uint8 pools of head_dim/2
    bytes per row (block_stride in bytes) and kv_scales uint8
    [num_blocks][2][Hkv][block_size][D/16]."""
    return _append_rows("paged_kv_append_rope_fp4", q_out, q, k_new, v_new, k_pool, v_pool, kv_scales, k_scale, v_scale,
                        block_table, positions, counts, cos_sin, rotary_dim, interleaved, q_norm, k_norm, eps,
                        block_size, num_blocks, block_stride, err_word, stream, prepare)


def paged_kv_append_fp4(k_new, v_new, k_pool, v_pool, kv_scales, block_table, positions, *, counts=None, k_scale=1.0,
                        v_scale=1.0, block_size, num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    """Quantising append of k_new/v_new [B][Hkv][D] or [B][T][Hkv][D] into the
    4-bit cache, as they are."""
    return _append_rows("paged_kv_append_fp4", None, None, k_new, v_new, k_pool, v_pool, kv_scales, k_scale, v_scale,
                        block_table, positions, counts, None, None, False, None, None, 0.0, block_size, num_blocks,
                        block_stride, err_word, stream, prepare)


def paged_kv_gather_fp4(k_out, v_out, k_pool, v_pool, kv_scales, block_table, starts, counts=None, *, k_scale=1.0,
                        v_scale=1.0, block_size, num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    """Values of tokens starts[b] + t, t < counts[b] (None: all T), of the 4-bit
    cache into k_out, v_out [B][T][Hkv][D]."""
    B, T, Hkv, D = k_out.shape
    dt = k_out.dtype
    if v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out differ in shape")
    _dense("k_out and v_out", dt, k_out, v_out)
    _dense("kv_scales", torch.uint8, kv_scales)
    _dense("block_table and starts", torch.int32, block_table, starts)
    rows, MB = block_table.shape
    if rows != B or starts.numel() != B:
        raise ValueError("block_table and starts must have one row per sequence")
    if counts is not None and not (counts.dtype == torch.int32 and counts.is_contiguous() and counts.numel() == B):
        raise ValueError("counts must be a contiguous torch.int32 tensor with one entry per sequence")
    if k_pool.dtype != torch.uint8 or v_pool.dtype != torch.uint8:
        raise ValueError("the pools must be uint8")
    _pools_hold(k_pool, v_pool, kv_scales, Hkv, D, block_size, num_blocks, block_stride)
    on = _launch_stream(stream, "paged_kv_gather_fp4", k_out, v_out, k_pool, v_pool, kv_scales, block_table, starts,
                        counts, err_word)
    shape = _SHAPE.pack(B, Hkv, Hkv, D, block_size, MB, num_blocks, block_stride, dtype_code(dt))
    args = (shape, k_out.data_ptr(), v_out.data_ptr(), T, k_pool.data_ptr(), v_pool.data_ptr(), kv_scales.data_ptr(),
            k_scale, v_scale, block_table.data_ptr(), starts.data_ptr(), _addr(counts), _addr(err_word), on)
    return _issue(load().paged_kv_gather_fp4, args, "paged_kv_gather_fp4", prepare)


def paged_attention_fp4_workspace(shape: Shape) -> int:
    return int(load().paged_attention_fp4_workspace(ctypes.byref(shape)))


def fp4_workspace_for(q, block_table, *, num_kv_heads, block_size, num_blocks, block_stride) -> torch.Tensor:
    """Allocate (through torch) a zero-filled workspace for
    paged_attention_decode_fp4 on q's device."""
    shape = decode_shape(q, block_table, num_kv_heads=num_kv_heads, block_size=block_size, num_blocks=num_blocks,
                         block_stride=block_stride)
    with torch.cuda.device(q.device):
        n = paged_attention_fp4_workspace(shape)
    if n == 0:
        raise PagedAttnError(PA_ERR_UNSUPPORTED, "paged_attention_fp4_workspace")
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=q.device)


def paged_attention_decode_fp4(out, q, k_pool, v_pool, kv_scales, block_table, seq_lens, scale, workspace, *,
                               k_scale=1.0, v_scale=1.0, window=0, num_kv_heads, block_size, num_blocks, block_stride,
                               err_word=None, stream=None, prepare=False):
    """out[B][H][D] = attention of q over the valid tokens (the last `window` of
    them when positive) of a 4-bit cache; workspace from fp4_workspace_for."""
    B, H, D = q.shape
    dt = q.dtype
    if out.shape != q.shape:
        raise ValueError("out and q differ in shape")
    _dense("q and out", dt, q, out)
    _dense("kv_scales and workspace", torch.uint8, kv_scales, workspace)
    _dense("block_table and seq_lens", torch.int32, block_table, seq_lens)
    rows, MB = block_table.shape
    if rows != B or seq_lens.numel() != B:
        raise ValueError("block_table and seq_lens must have one row per sequence")
    if k_pool.dtype != torch.uint8 or v_pool.dtype != torch.uint8:
        raise ValueError("the pools must be uint8")
    _pools_hold(k_pool, v_pool, kv_scales, num_kv_heads, D, block_size, num_blocks, block_stride)
    on = _launch_stream(stream, "paged_attention_decode_fp4", q, out, k_pool, v_pool, kv_scales, block_table, seq_lens,
                        workspace, err_word)
    shape = _SHAPE.pack(B, H, num_kv_heads, D, block_size, MB, num_blocks, block_stride, dtype_code(dt))
    args = (shape, out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), kv_scales.data_ptr(), k_scale,
            v_scale, block_table.data_ptr(), seq_lens.data_ptr(), scale, window, workspace.data_ptr(), workspace.numel(),
            _addr(err_word), on)
    return _issue(load().paged_attention_decode_fp4, args, "paged_attention_decode_fp4", prepare)


# ---------------------------------------------------------------------------
# attention of several new tokens per sequence
# ---------------------------------------------------------------------------

def paged_attention_chunk_workspace(shape: Shape) -> int:
    return int(load().paged_attention_chunk_workspace(ctypes.byref(shape)))


def chunk_workspace_for(q, block_table, *, num_kv_heads, block_size, num_blocks, block_stride) -> torch.Tensor:
    """Allocate (through torch) a workspace for paged_attention_chunk and
    paged_attention_chunk_diff on q's device; q is [B][H][D] or [B][T][H][D]."""
    shape = make_shape(batch=q.shape[0], num_heads=q.shape[-2], num_kv_heads=num_kv_heads, head_dim=q.shape[-1],
                       block_size=block_size, max_blocks_per_seq=block_table.shape[1], num_blocks=num_blocks,
                       block_stride=block_stride, dtype=q.dtype)
    with torch.cuda.device(q.device):
        n = paged_attention_chunk_workspace(shape)
    if n == 0:
        raise PagedAttnError(PA_ERR_UNSUPPORTED, "paged_attention_chunk_workspace")
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=q.device)


def _attend_rows(name, out, q, k_pool, v_pool, block_table, positions, scale, workspace, counts, window, num_kv_heads,
                 block_size, num_blocks, block_stride, err_word, stream, prepare, lambdas=None, norm=None, eps=0.0,
                 out_scale=1.0):
    dt = q.dtype
    B, T, H, D, qs = _new_rows("q", q)
    if out.numel() != B * T * H * D or out.dtype != dt or not out.is_contiguous():
        raise ValueError(f"out must be contiguous, with batch * tokens * heads * head_dim elements of {dt}")
    _dense("block_table and positions", torch.int32, block_table, positions)
    rows, MB = block_table.shape
    if rows != B or positions.numel() != B:
        raise ValueError("block_table and positions must have one row per sequence")
    if counts is not None and not (counts.dtype == torch.int32 and counts.is_contiguous() and counts.numel() == B):
        raise ValueError("counts must be a contiguous torch.int32 tensor with one entry per sequence")
    _dense("workspace", torch.uint8, workspace)
    if k_pool.dtype != dt or v_pool.dtype != dt:
        raise ValueError("the pools must be of the queries' dtype")
    _pools_hold(k_pool, v_pool, None, num_kv_heads, D, block_size, num_blocks, block_stride)
    diff = name == "paged_attention_chunk_diff"
    if diff and lambdas is None:
        raise ValueError("the differential form needs lambdas, one per head")
    on = _launch_stream(stream, name, q, out, k_pool, v_pool, block_table, positions, counts, workspace, err_word,
                        lambdas, norm)
    shape = _SHAPE.pack(B, H, num_kv_heads, D, block_size, MB, num_blocks, block_stride, dtype_code(dt))
    args = (out.data_ptr(), q.data_ptr(), qs, T, k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
            positions.data_ptr(), _addr(counts), scale, window, workspace.data_ptr(), workspace.numel(), _addr(err_word),
            on)
    if not diff:
        return _issue(load().paged_attention_chunk, (shape, *args), name, prepare)
    if lambdas.dtype != torch.float32 or not lambdas.is_contiguous() or lambdas.numel() != H:
        raise ValueError("lambdas must hold one contiguous torch.float32 element per head")
    if norm is not None and not (norm.dtype == dt and norm.is_contiguous() and norm.numel() == D):
        raise ValueError(f"norm must hold head_dim contiguous elements of {dt}")
    diff = _DIFF.pack(lambdas.data_ptr(), _addr(norm) or 0, eps, out_scale)
    return _issue(load().paged_attention_chunk_diff, (shape, diff, *args), name, prepare)


def paged_attention_chunk(out, q, k_pool, v_pool, block_table, positions, scale, workspace, *, counts=None, window=0,
                          num_kv_heads, block_size, num_blocks, block_stride, err_word=None, stream=None, prepare=False):
    """out[B][T][H][D] = attention of the new tokens' queries q ([B][H][D] or
    [B][T][H][D], a slice of a packed projection output included) over the
    cache: token t < counts[b] (None: all T) of sequence b sees positions up to
    its own, positions[b] + t (the last `window` of them when positive).
    Workspace from chunk_workspace_for."""
    return _attend_rows("paged_attention_chunk", out, q, k_pool, v_pool, block_table, positions, scale, workspace, counts,
                        window, num_kv_heads, block_size, num_blocks, block_stride, err_word, stream, prepare)


def paged_attention_chunk_diff(out, q, k_pool, v_pool, block_table, positions, lambdas, scale, workspace, *, counts=None,
                               norm=None, eps=1e-5, out_scale=1.0, window=0, num_kv_heads, block_size, num_blocks,
                               block_stride, err_word=None, stream=None, prepare=False):
    """paged_attention_chunk with the difference of two softmax maps (queries and
    keys of the first map in the first half of a row, of the second in the
    second): (softmax1 - lambdas[h] softmax2) V, then the norm over the head
    with weight norm [D] (None: none) and out_scale."""
    return _attend_rows("paged_attention_chunk_diff", out, q, k_pool, v_pool, block_table, positions, scale, workspace,
                        counts, window, num_kv_heads, block_size, num_blocks, block_stride, err_word, stream, prepare,
                        lambdas, norm, eps, out_scale)

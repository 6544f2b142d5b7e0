"""Python binding of libsbt.so (bounds-checked tile movement and the boundary-tile GEMM).

Argument marshalling only: every op runs in the library's CUDA kernels on the
caller's current torch stream.  torch supplies device memory and streams.
There is no fallback: if ``libsbt.so`` is missing or fails to load, importing
an op raises.

Op names match the C ABI in ``include/sbt.h`` without the ``sbt_`` prefix:
``tile_load_padded``, ``tile_store_clipped``, ``gather_rows``, ``gather_cols``,
``scatter_rows_masked``, ``scatter_add_rows``, ``ragged_tile_load``, ``ragged_tile_store``, ``gemm_bounded`` (plus
``gemm_bounded_workspace_size``), ``gemm_bounded_noalloc``, ``gemm_block_scaled`` (plus
``gemm_block_scaled_workspace_size``); of the paged cache and the layer around it ``paged_attention``,
``paged_tree_attention``, ``rope_table``, ``qk_norm_rope``, ``tree_plan``, ``pages_*``, ``add_rms_norm`` and
``matvec_e2m1``, gradients and workspace sizes beside them.  Arrays are torch tensors on the device
(only their data pointer is used; shapes and strides are the explicit
arguments, in elements).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsbt.so")

SBT_OK, SBT_ERR_INVALID_ARG, SBT_ERR_UNSUPPORTED, SBT_ERR_ALIGNMENT = 0, 1, 2, 3
SBT_ERR_TENSOR_MAP, SBT_ERR_CUDA, SBT_ERR_DEVICE_TIMEOUT = 4, 5, 6
STATUS_NAMES = {0: "SBT_OK", 1: "SBT_ERR_INVALID_ARG", 2: "SBT_ERR_UNSUPPORTED", 3: "SBT_ERR_ALIGNMENT",
                4: "SBT_ERR_TENSOR_MAP", 5: "SBT_ERR_CUDA", 6: "SBT_ERR_DEVICE_TIMEOUT"}
SBT_F32, SBT_BF16, SBT_F16 = 0, 1, 2
PATHS = {"auto": 0, "scalar": 1, "vector": 2, "tma": 3}

# Every symbol include/sbt.h declares.
EXPORTS = ("sbt_create", "sbt_destroy", "sbt_set_path", "sbt_set_wait_limit_ns", "sbt_set_test_hook", "sbt_launch_count",
           "sbt_check_status", "sbt_last_error_message", "sbt_tile_load_padded", "sbt_tile_store_clipped",
           "sbt_gather_rows", "sbt_gather_cols", "sbt_scatter_rows_masked", "sbt_scatter_add_rows", "sbt_ragged_tile_load", "sbt_ragged_tile_store", "sbt_gemm_bounded_workspace_size",
           "sbt_gemm_bounded", "sbt_gemm_block_scaled_workspace_size", "sbt_gemm_block_scaled",
           "sbt_gemm_bounded_noalloc", "sbt_paged_attention_workspace_size", "sbt_paged_attention", "sbt_rope_table",
           "sbt_qk_norm_rope", "sbt_qk_norm_rope_backward_workspace_size", "sbt_qk_norm_rope_backward",
           "sbt_pages_workspace_size", "sbt_pages_copy", "sbt_pages_reserve", "sbt_pages_fork", "sbt_pages_free",
           "sbt_pages_compact", "sbt_pages_slots", "sbt_tree_plan", "sbt_paged_tree_attention_workspace_size",
           "sbt_paged_tree_attention", "sbt_add_rms_norm", "sbt_add_rms_norm_backward_workspace_size",
           "sbt_add_rms_norm_backward", "sbt_matvec_e2m1")
LOWP_FORMATS = {"e4m3": 0, "e5m2": 1, "e8m0": 2, "e2m1": 3}  # sbt_lowp_format
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}  # sbt_rope_layout
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}  # sbt_rope_scaling
MAX_PAGE_POOLS = 64  # SBT_MAX_PAGE_POOLS in include/sbt.h
GEMM_NOALLOC_SCRATCH_BYTES = 16 << 20  # SBT_GEMM_NOALLOC_SCRATCH_BYTES in include/sbt.h


class SbtError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class KvCache(ctypes.Structure):
    """``sbt_kv_cache``: keys and values of one layer in pages (made by ``kv_cache``)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("ld_page", ctypes.c_int64), ("ld_slot", ctypes.c_int64),
                ("ld_head", ctypes.c_int64)]


class PageMap(ctypes.Structure):
    """``sbt_page_map``: the sequences' pages, lengths and the pages' holders (made by ``page_map``)."""
    _fields_ = [("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("n_seq", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("lens", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("refs", ctypes.c_void_p)]


class Rope(ctypes.Structure):
    """``sbt_rope``: a table of rotations and which elements they turn (made by ``rope``)."""
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32)]


class PagePool(ctypes.Structure):
    """``sbt_page_pool`` (arrays of them are made by ``page_pools``)."""
    _fields_ = [("base", ctypes.c_void_p), ("n_planes", ctypes.c_int64), ("plane_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64)]


class CodeRows(ctypes.Structure):
    """``sbt_code_rows``: 8-bit codes and their scales (made by ``code_rows``)."""
    _fields_ = [("codes", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("ld_scale", ctypes.c_int64), ("format", ctypes.c_int32), ("block", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH):
    """Load libsbt.so and declare its signatures (no CUDA call is made)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libsbt.so not built ({path}); run `python -m scatter_boundary_tile_gb300._build`")
        lib = ctypes.CDLL(path)
        p, i64, i32, u64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_int
        sig = {
            "sbt_create": [ci, ctypes.POINTER(p)],
            "sbt_destroy": [p],
            "sbt_set_path": [p, ci],
            "sbt_set_wait_limit_ns": [p, u64],
            "sbt_set_test_hook": [p, ci],
            "sbt_check_status": [p, p],
            "sbt_tile_load_padded": [p, ci, p, i64, i64, i64, i64, i64, i64, i64, i64, i32, i32, i32, i32, p, p, p],
            "sbt_tile_store_clipped": [p, ci, p, i32, i32, i32, i32, p, i64, i64, i64, i64, i64, i64, i64, i64, p],
            "sbt_gather_rows": [p, ci, p, i64, i64, i64, p, i64, i64, i64, i32, p, i64, p, i64, p, p],
            "sbt_scatter_rows_masked": [p, ci, p, i64, i64, i64, p, i64, i64, i64, p, i64, i32, p, i64, p],
            "sbt_gather_cols": [p, ci, p, i64, i64, i64, p, i64, i64, i64, i32, p, i64, p, p],
            "sbt_scatter_add_rows": [p, ci, p, i64, i64, i64, p, i64, i64, i64, p, i64, i32, p],
            "sbt_ragged_tile_load": [p, ci, p, i64, i32, i32, i64, i64, p, i32, i32, p, p],
            "sbt_ragged_tile_store": [p, ci, p, i32, i32, i32, i32, p, p, i64, i64, i64, p],
            "sbt_gemm_bounded_workspace_size": [p, i64, i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)],
            "sbt_gemm_bounded": [p, p, i64, p, i64, p, i64, ci, i64, i64, i64, p, ctypes.c_size_t, p],
            "sbt_gemm_bounded_noalloc": [p, p, i64, p, i64, p, i64, ci, i64, i64, i64, p],
            "sbt_gemm_block_scaled_workspace_size": [p, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)],
            "sbt_gemm_block_scaled": [p, ci, p, i64, ci, p, i64, ci, p, i64, p, i64, i64, p, i64, p, i64, i64, i64,
                                      i64, p, ctypes.c_size_t, p],
        }
        pp, sz, f32, f64 = ctypes.POINTER, ctypes.c_size_t, ctypes.c_float, ctypes.c_double
        cache, pmap, turn, pool = pp(KvCache), pp(PageMap), pp(Rope), pp(PagePool)
        rows = [p, i64, i64]
        sig.update({
            "sbt_paged_attention_workspace_size": [p, i32, i32, i32, pp(sz)],
            "sbt_paged_attention": [p, ci, *rows, i32, i32, cache, pmap, p, f32, i32, *rows, p, p, sz, p],
            "sbt_rope_table": [p, p, i64, i32, f64, ci, f64, i64, f64, f64, f64, p],
            "sbt_qk_norm_rope": [p, ci, *rows, *rows, i64, i32, i32, i32, p, turn, p, p, f32, *rows, *rows, *rows,
                                 cache, pmap, p, p],
            "sbt_qk_norm_rope_backward_workspace_size": [p, i32, pp(sz)],
            "sbt_qk_norm_rope_backward": [p, ci, *rows, *rows, *rows, *rows, i64, i32, i32, i32, p, turn, p, p, f32,
                                          *rows, *rows, p, p, p, sz, p],
            "sbt_pages_workspace_size": [p, i32, i64, pp(sz)],
            "sbt_pages_copy": [p, pool, i32, i64, p, p, i64, p],
            "sbt_pages_reserve": [p, pmap, pool, i32, p, p, sz, p],
            "sbt_pages_fork": [p, pmap, pool, i32, p, p, i32, p, sz, p],
            "sbt_pages_free": [p, pmap, p, p, i32, p],
            "sbt_pages_compact": [p, pmap, pool, i32, p, i64, p, p, p, p, sz, p],
            "sbt_pages_slots": [p, pmap, p, i32, p, p, i32, p, p, p, p, p, p],
            "sbt_tree_plan": [p, p, p, i32, i32, p, p, p, i64, p],
            "sbt_paged_tree_attention_workspace_size": [p, i32, i32, i32, i32, pp(sz)],
            "sbt_paged_tree_attention": [p, ci, *rows, i32, p, i32, i32, i32, cache, pmap, p, f32, p, i64, *rows, p, p,
                                         sz, p],
            "sbt_add_rms_norm": [p, ci, p, i64, p, i64, i64, i32, p, f32, p, i64, p, i64, pp(CodeRows), p],
            "sbt_add_rms_norm_backward_workspace_size": [p, i64, i32, pp(sz)],
            "sbt_add_rms_norm_backward": [p, ci, p, i64, p, i64, p, i64, i64, i32, p, f32, p, i64, p, p, sz, p],
            "sbt_matvec_e2m1": [p, ci, p, i64, i64, p, i64, ci, p, i64, i64, f32, p, i64, ci, i64, i64, p],
        })
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = ci
        lib.sbt_launch_count.argtypes = [p]
        lib.sbt_launch_count.restype = u64
        lib.sbt_last_error_message.argtypes = []
        lib.sbt_last_error_message.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(status: int):
    if status != SBT_OK:
        msg = load_library().sbt_last_error_message().decode(errors="replace")
        raise SbtError(status, msg)


def _ptr(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


_torch = None  # the torch module, its raw-stream query and its dtypes' codes, once a call needs them


def _load_torch():
    global _torch, _raw_stream, _device_index, _CODES
    import torch
    _device_index = torch.cuda.current_device
    # not a public name of torch: without it a Stream object is built per call
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:
        _raw_stream = lambda device: torch.cuda.current_stream(device).cuda_stream
    _CODES = {torch.float32: SBT_F32, torch.bfloat16: SBT_BF16, torch.float16: SBT_F16}
    _torch = torch


def _stream(stream) -> int | None:
    if stream is None:  # the current device's current stream, without building a Stream object
        if _torch is None:
            _load_torch()
        return _raw_stream(_device_index())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t, dtype):
    if dtype is not None:
        return {"f32": SBT_F32, "bf16": SBT_BF16, "f16": SBT_F16}[dtype] if isinstance(dtype, str) else int(dtype)
    if _torch is None:
        _load_torch()
    code = _CODES.get(t.dtype)
    return {4: SBT_F32, 2: SBT_BF16}[t.element_size()] if code is None else code


def _pad_bytes(pad, code):
    """One element's bits: an int is taken as raw bits, a float is converted to the dtype."""
    if pad is None:
        return None
    if isinstance(pad, (bytes, bytearray)):
        return ctypes.create_string_buffer(bytes(pad), len(pad))
    if code == SBT_F32:
        raw = struct.pack("<I", pad & 0xFFFFFFFF) if isinstance(pad, int) else struct.pack("<f", pad)
    else:
        if isinstance(pad, int):
            raw = struct.pack("<H", pad & 0xFFFF)
        else:
            import torch
            tdt = torch.bfloat16 if code == SBT_BF16 else torch.float16
            bits = torch.tensor([float(pad)], dtype=torch.float32).to(tdt).view(torch.int16).item()
            raw = struct.pack("<H", bits & 0xFFFF)
    return ctypes.create_string_buffer(raw, len(raw))


class Context:
    """An ``sbt_context`` bound to one CUDA device."""

    def __init__(self, device: int = 0):
        lib = load_library()
        h = ctypes.c_void_p()
        _check(lib.sbt_create(device, ctypes.byref(h)))
        self._h = h
        self.device = device

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load_library().sbt_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_path(self, path: str):
        _check(load_library().sbt_set_path(self._h, PATHS[path]))

    def set_wait_limit_ns(self, ns: int):
        _check(load_library().sbt_set_wait_limit_ns(self._h, ns))

    def set_test_hook(self, withhold_load: bool):
        """Test only: make the next GEMM / bulk row launches withhold their first copy."""
        _check(load_library().sbt_set_test_hook(self._h, 1 if withhold_load else 0))

    @property
    def launch_count(self) -> int:
        return int(load_library().sbt_launch_count(self._h))

    def check_status(self, stream=None):
        _check(load_library().sbt_check_status(self._h, _stream(stream)))


def tile_load_padded(ctx, src, rows, cols, stride_r, stride_c, origin_r, origin_c, step_r, step_c, grid_r, grid_c,
                     tile_r, tile_c, dst_tiles, pad=None, dtype=None, stream=None):
    code = _dtype_code(dst_tiles, dtype)
    _check(load_library().sbt_tile_load_padded(ctx.handle, code, _ptr(src), rows, cols, stride_r, stride_c, origin_r,
                                               origin_c, step_r, step_c, grid_r, grid_c, tile_r, tile_c,
                                               _ptr(dst_tiles), _pad_bytes(pad, code), _stream(stream)))


def tile_store_clipped(ctx, src_tiles, grid_r, grid_c, tile_r, tile_c, dst, rows, cols, stride_r, stride_c, origin_r,
                       origin_c, step_r, step_c, dtype=None, stream=None):
    code = _dtype_code(src_tiles, dtype)
    _check(load_library().sbt_tile_store_clipped(ctx.handle, code, _ptr(src_tiles), grid_r, grid_c, tile_r, tile_c,
                                                 _ptr(dst), rows, cols, stride_r, stride_c, origin_r, origin_c,
                                                 step_r, step_c, _stream(stream)))


def gather_rows(ctx, src, rows, cols, ld_src, idx, n_idx, out, ld_out, tile_c, row_offset=0, col_offset=0,
                mask=None, ld_mask=0, pad=None, dtype=None, stream=None):
    code = _dtype_code(out, dtype)
    _check(load_library().sbt_gather_rows(ctx.handle, code, _ptr(src), rows, cols, ld_src, _ptr(idx), n_idx,
                                          row_offset, col_offset, tile_c, _ptr(mask), ld_mask, _ptr(out), ld_out,
                                          _pad_bytes(pad, code), _stream(stream)))


def gather_cols(ctx, src, rows, cols, ld_src, idx, n_idx, out, ld_out, tile_r, row_offset=0, col_offset=0, pad=None,
                dtype=None, stream=None):
    code = _dtype_code(out, dtype)
    _check(load_library().sbt_gather_cols(ctx.handle, code, _ptr(src), rows, cols, ld_src, _ptr(idx), n_idx, row_offset,
                                          col_offset, tile_r, _ptr(out), ld_out, _pad_bytes(pad, code),
                                          _stream(stream)))


def scatter_rows_masked(ctx, dst, rows, cols, ld_dst, idx, n_idx, src, ld_src, tile_c, row_offset=0, col_offset=0,
                        mask=None, ld_mask=0, dtype=None, stream=None):
    code = _dtype_code(dst, dtype)
    _check(load_library().sbt_scatter_rows_masked(ctx.handle, code, _ptr(dst), rows, cols, ld_dst, _ptr(idx), n_idx,
                                                  row_offset, col_offset, _ptr(src), ld_src, tile_c, _ptr(mask),
                                                  ld_mask, _stream(stream)))


def scatter_add_rows(ctx, dst, rows, cols, ld_dst, idx, n_idx, src, ld_src, tile_c, row_offset=0, col_offset=0,
                     dtype=None, stream=None):
    code = _dtype_code(dst, dtype)
    _check(load_library().sbt_scatter_add_rows(ctx.handle, code, _ptr(dst), rows, cols, ld_dst, _ptr(idx), n_idx,
                                               row_offset, col_offset, _ptr(src), ld_src, tile_c, _stream(stream)))


def ragged_tile_load(ctx, x, total_rows, heads, depth, ld_row, ld_head, cu_seqlens, batch, t_pad, out, dtype=None,
                     stream=None):
    code = _dtype_code(out, dtype)
    _check(load_library().sbt_ragged_tile_load(ctx.handle, code, _ptr(x), total_rows, heads, depth, ld_row, ld_head,
                                               _ptr(cu_seqlens), batch, t_pad, _ptr(out), _stream(stream)))


def ragged_tile_store(ctx, tiles, batch, heads, depth, t_pad, cu_seqlens, x, total_rows, ld_row, ld_head, dtype=None,
                      stream=None):
    code = _dtype_code(tiles, dtype)
    _check(load_library().sbt_ragged_tile_store(ctx.handle, code, _ptr(tiles), batch, heads, depth, t_pad,
                                                _ptr(cu_seqlens), _ptr(x), total_rows, ld_row, ld_head,
                                                _stream(stream)))


def gemm_bounded_workspace_size(ctx, M, N, K, lda, ldb) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_gemm_bounded_workspace_size(ctx.handle, M, N, K, lda, ldb, ctypes.byref(n)))
    return int(n.value)


def gemm_bounded(ctx, A, lda, B, ldb, C, ldc, M, N, K, workspace=None, workspace_bytes=0, c_dtype="bf16",
                 stream=None):
    code = {"bf16": SBT_BF16, "f32": SBT_F32}[c_dtype] if isinstance(c_dtype, str) else int(c_dtype)
    _check(load_library().sbt_gemm_bounded(ctx.handle, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, code, M, N, K,
                                           _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_block_scaled_workspace_size(ctx, M, N, K) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_gemm_block_scaled_workspace_size(ctx.handle, M, N, K, ctypes.byref(n)))
    return int(n.value)


def gemm_block_scaled(ctx, A, lda, B, ldb, a_scale, ld_sa, b_scale, ld_sb, K_s, D, ldd, M, N, K, acc=None, ld_acc=0,
                      workspace=None, workspace_bytes=0, a_fmt="e4m3", b_fmt="e4m3", s_fmt="e8m0", stream=None):
    """sbt_gemm_block_scaled: D = (A .* a_scale)(B .* b_scale) + acc; formats by name (see LOWP_FORMATS)."""
    fmt = lambda f: LOWP_FORMATS[f] if isinstance(f, str) else int(f)
    _check(load_library().sbt_gemm_block_scaled(ctx.handle, fmt(a_fmt), _ptr(A), lda, fmt(b_fmt), _ptr(B), ldb,
                                                fmt(s_fmt), _ptr(a_scale), ld_sa, _ptr(b_scale), ld_sb, K_s,
                                                _ptr(acc), ld_acc, _ptr(D), ldd, M, N, K, _ptr(workspace),
                                                workspace_bytes, _stream(stream)))


def gemm_bounded_noalloc(ctx, A, lda, B, ldb, C, ldc, M, N, K, c_dtype="bf16", stream=None):
    """sbt_gemm_bounded_noalloc: the bounded GEMM with the library's fixed staging scratch.

    For callers that cannot allocate device memory at the call: plugins
    confined to another framework's memory pool, code under a device-memory
    budget committed up front, or paths that cannot take cudaMalloc's implicit
    synchronisation.  Shapes needing more than GEMM_NOALLOC_SCRATCH_BYTES of
    staging are rejected; calls that may overlap on the GPU race on the shared
    scratch.
    """
    code = {"bf16": SBT_BF16, "f32": SBT_F32}[c_dtype] if isinstance(c_dtype, str) else int(c_dtype)
    _check(load_library().sbt_gemm_bounded_noalloc(ctx.handle, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, code, M, N,
                                                   K, _stream(stream)))


# --------------------------------------------------------------------------- paged key-value cache
# The handles below are plain structs of addresses and sizes, made once and passed to every call;
# they keep the tensors they were made of alive.

def kv_cache(k, v, heads, head_dim, ld_page, ld_slot, ld_head) -> KvCache:
    """sbt_kv_cache: element (page, slot, head, d) at page*ld_page + slot*ld_slot + head*ld_head + d of k and of v."""
    c = KvCache(_ptr(k), _ptr(v), heads, head_dim, ld_page, ld_slot, ld_head)
    c.tensors = (k, v)
    return c


def page_map(page_table, ld_table, n_seq, max_pages, lens, n_pages, page_size, refs=None) -> PageMap:
    """sbt_page_map: int32 page_table [n_seq][ld_table], lens [n_seq] and refs [n_pages] (where a call needs them)."""
    m = PageMap(_ptr(page_table), ld_table, n_seq, max_pages, _ptr(lens), n_pages, page_size, _ptr(refs))
    m.tensors = (page_table, lens, refs)
    return m


def rope(table, n_pos, rot_dim, layout="half") -> Rope:
    """sbt_rope: fp32 table [n_pos][rot_dim/2][2] of (cos, sin), as rope_table fills it."""
    r = Rope(_ptr(table), n_pos, rot_dim, ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout))
    r.tensors = (table,)
    return r


def page_pools(pools):
    """Array of sbt_page_pool from tuples (base, n_planes, plane_stride, page_stride, page_bytes), in bytes."""
    a = (PagePool * len(pools))(*[PagePool(_ptr(b), n, ps, gs, nb) for b, n, ps, gs, nb in pools])
    a.tensors = tuple(t[0] for t in pools)
    return a


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def paged_attention_workspace_size(ctx, q_heads, kv_heads, head_dim) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_paged_attention_workspace_size(ctx.handle, q_heads, kv_heads, head_dim, ctypes.byref(n)))
    return int(n.value)


def paged_attention(ctx, q, ld_q, ld_qh, batch, q_heads, cache, map, scale, out, ld_out, ld_oh, lse=None, window=0,
                    seq=None, workspace=None, workspace_bytes=0, dtype=None, stream=None):
    """sbt_paged_attention: one new token per batch entry over the first lens positions of its sequence."""
    code = _dtype_code(q, dtype)
    _check(load_library().sbt_paged_attention(ctx.handle, code, _ptr(q), ld_q, ld_qh, batch, q_heads, _ref(cache),
                                              _ref(map), _ptr(seq), scale, window, _ptr(out), ld_out, ld_oh, _ptr(lse),
                                              _ptr(workspace), workspace_bytes, _stream(stream)))


def rope_table(ctx, table, n_pos, rot_dim, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=1.0, high=32.0,
               amplitude=1.0, stream=None):
    """sbt_rope_table: fills the fp32 table [n_pos][rot_dim/2][2]; scalings by name (see ROPE_SCALINGS)."""
    code = ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    _check(load_library().sbt_rope_table(ctx.handle, _ptr(table), n_pos, rot_dim, base, code, factor, orig_len, low,
                                         high, amplitude, _stream(stream)))


def qk_norm_rope(ctx, q, ld_q, ld_qh, k, ld_k, ld_kh, tokens, q_heads, k_heads, head_dim, positions, rope, q_out,
                 ld_qo, ld_qoh, k_out=None, ld_ko=0, ld_koh=0, q_weight=None, k_weight=None, eps=1e-6, v=None, ld_v=0,
                 ld_vh=0, cache=None, map=None, seq=None, dtype=None, stream=None):
    """sbt_qk_norm_rope: norm and rotation of q and k; with a cache, k and v are appended at `positions`."""
    code = _dtype_code(k if q is None else q, dtype)
    _check(load_library().sbt_qk_norm_rope(ctx.handle, code, _ptr(q), ld_q, ld_qh, _ptr(k), ld_k, ld_kh, tokens,
                                           q_heads, k_heads, head_dim, _ptr(positions), _ref(rope), _ptr(q_weight),
                                           _ptr(k_weight), eps, _ptr(q_out), ld_qo, ld_qoh, _ptr(k_out), ld_ko, ld_koh,
                                           _ptr(v), ld_v, ld_vh, _ref(cache), _ref(map), _ptr(seq), _stream(stream)))


def qk_norm_rope_backward_workspace_size(ctx, head_dim) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_qk_norm_rope_backward_workspace_size(ctx.handle, head_dim, ctypes.byref(n)))
    return int(n.value)


def qk_norm_rope_backward(ctx, gq, ld_gq, ld_gqh, gk, ld_gk, ld_gkh, q, ld_q, ld_qh, k, ld_k, ld_kh, tokens, q_heads,
                          k_heads, head_dim, positions, rope, dq, ld_dq, ld_dqh, dk, ld_dk, ld_dkh, q_weight=None,
                          k_weight=None, eps=1e-6, dq_weight=None, dk_weight=None, workspace=None, workspace_bytes=0,
                          dtype=None, stream=None):
    """sbt_qk_norm_rope_backward: gradients of q and k (and, fp32, of the weights) from those of q_out and k_out."""
    code = _dtype_code(gk if gq is None else gq, dtype)
    _check(load_library().sbt_qk_norm_rope_backward(
        ctx.handle, code, _ptr(gq), ld_gq, ld_gqh, _ptr(gk), ld_gk, ld_gkh, _ptr(q), ld_q, ld_qh, _ptr(k), ld_k, ld_kh,
        tokens, q_heads, k_heads, head_dim, _ptr(positions), _ref(rope), _ptr(q_weight), _ptr(k_weight), eps, _ptr(dq),
        ld_dq, ld_dqh, _ptr(dk), ld_dk, ld_dkh, _ptr(dq_weight), _ptr(dk_weight), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def pages_workspace_size(ctx, n_seq, n_pages) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_pages_workspace_size(ctx.handle, n_seq, n_pages, ctypes.byref(n)))
    return int(n.value)


def pages_copy(ctx, pools, n_pages, src, dst, n, stream=None):
    """sbt_pages_copy: page src[i] to page dst[i] in every plane of every pool."""
    _check(load_library().sbt_pages_copy(ctx.handle, pools, len(pools), n_pages, _ptr(src), _ptr(dst), n,
                                         _stream(stream)))


def pages_reserve(ctx, map, pools, target, workspace, workspace_bytes, stream=None):
    """sbt_pages_reserve: grow the sequences to target positions (map's lens show which did)."""
    _check(load_library().sbt_pages_reserve(ctx.handle, _ref(map), pools, len(pools), _ptr(target), _ptr(workspace),
                                            workspace_bytes, _stream(stream)))


def pages_fork(ctx, map, pools, from_seq, to_seq, n, workspace, workspace_bytes, stream=None):
    """sbt_pages_fork: sequence to_seq[i] becomes a copy of from_seq[i] that shares its full pages."""
    _check(load_library().sbt_pages_fork(ctx.handle, _ref(map), pools, len(pools), _ptr(from_seq), _ptr(to_seq), n,
                                         _ptr(workspace), workspace_bytes, _stream(stream)))


def pages_free(ctx, map, seqs, n, keep=None, stream=None):
    """sbt_pages_free: cut sequence seqs[i] to keep[i] positions (to none without keep)."""
    _check(load_library().sbt_pages_free(ctx.handle, _ref(map), _ptr(seqs), _ptr(keep), n, _stream(stream)))


def pages_compact(ctx, map, pools, table_out, ld_out, refs_out, page_to, n_live, workspace, workspace_bytes,
                  stream=None):
    """sbt_pages_compact: pack the held pages to the front; page_to gets every page's new number or -1."""
    _check(load_library().sbt_pages_compact(ctx.handle, _ref(map), pools, len(pools), _ptr(table_out), ld_out,
                                            _ptr(refs_out), _ptr(page_to), _ptr(n_live), _ptr(workspace),
                                            workspace_bytes, _stream(stream)))


def pages_slots(ctx, map, n_new, batch, capacity, seqs=None, start=None, cu=None, seq=None, positions=None, slots=None,
                last=None, stream=None):
    """sbt_pages_slots: prefix sums of n_new, and each new token's sequence, position and slot; -1 pads to capacity."""
    _check(load_library().sbt_pages_slots(ctx.handle, _ref(map), _ptr(n_new), batch, _ptr(seqs), _ptr(start), capacity,
                                          _ptr(cu), _ptr(seq), _ptr(positions), _ptr(slots), _ptr(last),
                                          _stream(stream)))


def tree_plan(ctx, parents, cu, batch, rows, mask=None, ld_mask=0, positions=None, turned=None, stream=None):
    """sbt_tree_plan: ancestor bits (int32 [rows][ld_mask]) and rotation positions of trees of drafted tokens."""
    _check(load_library().sbt_tree_plan(ctx.handle, _ptr(parents), _ptr(cu), batch, rows, _ptr(positions),
                                        _ptr(turned), _ptr(mask), ld_mask, _stream(stream)))


def paged_tree_attention_workspace_size(ctx, max_new, q_heads, kv_heads, head_dim) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_paged_tree_attention_workspace_size(ctx.handle, max_new, q_heads, kv_heads, head_dim,
                                                                  ctypes.byref(n)))
    return int(n.value)


def paged_tree_attention(ctx, q, ld_q, ld_qh, rows, cu, batch, max_new, q_heads, cache, map, scale, out, ld_out, ld_oh,
                         mask=None, ld_mask=0, lse=None, seq=None, workspace=None, workspace_bytes=0, dtype=None,
                         stream=None):
    """sbt_paged_tree_attention: rows cu[b] .. cu[b+1] - 1 are the last tokens of entry b's sequence (a tree or a chain)."""
    code = _dtype_code(q, dtype)
    _check(load_library().sbt_paged_tree_attention(ctx.handle, code, _ptr(q), ld_q, ld_qh, rows, _ptr(cu), batch,
                                                   max_new, q_heads, _ref(cache), _ref(map), _ptr(seq), scale,
                                                   _ptr(mask), ld_mask, _ptr(out), ld_out, ld_oh, _ptr(lse),
                                                   _ptr(workspace), workspace_bytes, _stream(stream)))


# --------------------------------------------------------------------------- around the attention

def code_rows(codes, ld, scales, ld_scale, fmt="e4m3", block=32) -> CodeRows:
    """sbt_code_rows: 8-bit codes [rows][ld] with an E8M0 scale per `block` columns [rows][ld_scale]."""
    c = CodeRows(_ptr(codes), ld, _ptr(scales), ld_scale, LOWP_FORMATS[fmt] if isinstance(fmt, str) else int(fmt), block)
    c.tensors = (codes, scales)
    return c


def add_rms_norm(ctx, x, ld_x, rows, cols, weight=None, eps=1e-6, r=None, ld_r=0, h_out=None, ld_h=0, y=None, ld_y=0,
                 codes=None, dtype=None, stream=None):
    """sbt_add_rms_norm: h = x + r and its RMS norm, as numbers (y) and as 8-bit codes with block scales (codes)."""
    code = _dtype_code(x, dtype)
    _check(load_library().sbt_add_rms_norm(ctx.handle, code, _ptr(x), ld_x, _ptr(r), ld_r, rows, cols, _ptr(weight),
                                           eps, _ptr(h_out), ld_h, _ptr(y), ld_y, _ref(codes), _stream(stream)))


def add_rms_norm_backward_workspace_size(ctx, rows, cols) -> int:
    n = ctypes.c_size_t()
    _check(load_library().sbt_add_rms_norm_backward_workspace_size(ctx.handle, rows, cols, ctypes.byref(n)))
    return int(n.value)


def add_rms_norm_backward(ctx, gy, ld_gy, h, ld_h, rows, cols, dx, ld_dx, gh=None, ld_gh=0, weight=None, eps=1e-6,
                          dweight=None, workspace=None, workspace_bytes=0, dtype=None, stream=None):
    """sbt_add_rms_norm_backward: gradient of x (and of r) from those of y and h_out, and, fp32, the weight's."""
    code = _dtype_code(gy, dtype)
    _check(load_library().sbt_add_rms_norm_backward(ctx.handle, code, _ptr(gy), ld_gy, _ptr(gh), ld_gh, _ptr(h), ld_h,
                                                    rows, cols, _ptr(weight), eps, _ptr(dx), ld_dx, _ptr(dweight),
                                                    _ptr(workspace), workspace_bytes, _stream(stream)))


def matvec_e2m1(ctx, x, ld_x, tokens, B, ldb, b_scale, ld_sb, K_s, y, ld_y, N, K, s_fmt="e8m0", alpha=1.0, dtype=None,
                y_dtype=None, stream=None):
    """sbt_matvec_e2m1: y = alpha * x (B .* b_scale) for a few tokens; B and b_scale as gemm_block_scaled takes them."""
    code, y_code = _dtype_code(x, dtype), _dtype_code(y, y_dtype)
    s = LOWP_FORMATS[s_fmt] if isinstance(s_fmt, str) else int(s_fmt)
    _check(load_library().sbt_matvec_e2m1(ctx.handle, code, _ptr(x), ld_x, tokens, _ptr(B), ldb, s, _ptr(b_scale),
                                          ld_sb, K_s, alpha, _ptr(y), ld_y, y_code, N, K, _stream(stream)))

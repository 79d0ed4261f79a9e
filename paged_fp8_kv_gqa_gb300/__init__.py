"""Python binding of libxqa: paged E5M2-KV grouped-query decode attention on sm_103a.

Argument marshalling only. Every step of the decode runs in the CUDA kernels of
``libxqa.so``; PyTorch supplies device memory and streams. There is no CPU
fallback: if the library is not built, or a tensor is not on a CUDA device,
these functions raise.

The names mirror the C ABI declared in ``include/xqa.h``:
``xqa_workspace_size``, ``xqa_decode``, ``xqa_plan``, ``xqa_attend_partial``,
``xqa_combine``, ``xqa_decode_device_scales``, ``xqa_dequant_e5m2``,
``xqa_dequant_e4m3``, ``xqa_read_status``, ``xqa_read_plan``, ``xqa_status_string``,
``xqa_decode_static_workspace``, ``xqa_kernels_per_call``, ``xqa_append``,
``xqa_gather``, ``xqa_prefill``, ``xqa_prefill_workspace_size``, ``xqa_extend``,
``xqa_extend_workspace_size``, ``xqa_assign_pages``, ``xqa_release_pages``,
``xqa_page_bounds``, ``xqa_select``, ``xqa_select_workspace_size``,
``xqa_decode_selected``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libxqa.so")

XQA_OK = 0
XQA_ERR_NULL = 1
XQA_ERR_SHAPE = 2
XQA_ERR_ALIGN = 3
XQA_ERR_WORKSPACE = 4
XQA_ERR_LAUNCH = 5
XQA_ERR_DEVICE = 6
XQA_ERR_VALUE = 7
XQA_ERR_BAD_BLOCK_ID = 16
XQA_ERR_CTX_TOO_LONG = 17
XQA_ERR_DEVICE_TIMEOUT = 18
XQA_ERR_DRAIN_TIMEOUT = 19
XQA_ERR_BAD_OFFSETS = 20
XQA_ERR_NO_PAGES = 21

#: C symbols the library exports (kept in step with include/xqa.h).
EXPORTED = (
    "xqa_workspace_size",
    "xqa_decode",
    "xqa_plan",
    "xqa_attend_partial",
    "xqa_combine",
    "xqa_dequant_e5m2",
    "xqa_read_status",
    "xqa_read_plan",
    "xqa_status_string",
    "xqa_decode_static_workspace",
    "xqa_decode_device_scales",
    "xqa_dequant_e4m3",
    "xqa_selftest_wait_timeout",
    "xqa_kernels_per_call",
    "xqa_append",
    "xqa_gather",
    "xqa_prefill",
    "xqa_prefill_workspace_size",
    "xqa_extend",
    "xqa_extend_workspace_size",
    "xqa_assign_pages",
    "xqa_release_pages",
    "xqa_page_bounds",
    "xqa_select",
    "xqa_select_workspace_size",
    "xqa_decode_selected",
)

KV_DTYPES = {"e5m2": 0, "e4m3": 1, "e2m1": 4}
KV_LAYOUTS = {"hnd": 0, "nhd": 1}
#: bytes of a (page, kv head) slice of a 4-bit cache (XQA_E2M1_SLICE_BYTES)
E2M1_SLICE_BYTES = 1152
#: bytes of a (page, kv head) slice of the bounds (XQA_BOUNDS_BYTES)
BOUNDS_BYTES = 272
ROW_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_F16, _U8, _I32 = torch.float16, torch.uint8, torch.int32


class XqaShape(ctypes.Structure):
    """Mirror of ``xqa_shape_t``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("sm_scale", ctypes.c_float),
        ("max_ctas", ctypes.c_int32),
        ("min_pages_per_cta", ctypes.c_int32),
        ("merge_mode", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("kv_layout", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
    ]


class XqaRows(ctypes.Structure):
    """Mirror of ``xqa_rows_t``."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_kv_heads", "head_dim", "block_size", "max_blocks_per_seq", "num_blocks",
        "num_rows", "kv_dtype", "kv_layout", "dtype")]
    _fields_ += [(n, ctypes.c_int64) for n in (
        "k_row_stride", "k_head_stride", "v_row_stride", "v_head_stride")]


class XqaPrefillShape(ctypes.Structure):
    """Mirror of ``xqa_prefill_shape_t``."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "total_q", "total_k", "dtype",
        "causal")]
    _fields_ += [("sm_scale", ctypes.c_float), ("max_ctas", ctypes.c_int32)]
    _fields_ += [(n, ctypes.c_int64) for n in (
        "q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride", "v_row_stride",
        "v_head_stride", "out_row_stride", "out_head_stride")]


class XqaExtendShape(ctypes.Structure):
    """Mirror of ``xqa_extend_shape_t``."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "block_size", "max_blocks_per_seq",
        "num_blocks", "total_q", "dtype", "kv_dtype", "kv_layout", "causal")]
    _fields_ += [("sm_scale", ctypes.c_float), ("max_ctas", ctypes.c_int32)]
    _fields_ += [(n, ctypes.c_int64) for n in (
        "q_row_stride", "q_head_stride", "out_row_stride", "out_head_stride")]


class XqaPages(ctypes.Structure):
    """Mirror of ``xqa_pages_t``."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "block_size", "max_blocks_per_seq", "num_blocks", "num_rows")]


class XqaSelectShape(ctypes.Structure):
    """Mirror of ``xqa_select_shape_t``."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "block_size", "max_blocks_per_seq",
        "num_blocks", "max_pages", "first_pages", "last_pages", "max_ctas")]


class XqaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {xqa_status_string(code)} (status {code})")


_lib = None

_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_SHAPE = ctypes.POINTER(XqaShape)
_DIMS_AT, _CAUSAL_AT = XqaPrefillShape.num_q_heads.offset, XqaPrefillShape.causal.offset
_STRIDES_AT, _OUT_AT = XqaPrefillShape.q_row_stride.offset, XqaPrefillShape.out_row_stride.offset
_ROWS = ctypes.POINTER(XqaRows)
_PREFILL = ctypes.POINTER(XqaPrefillShape)
_EXTEND = ctypes.POINTER(XqaExtendShape)
_PAGES = ctypes.POINTER(XqaPages)
_SELECT = ctypes.POINTER(XqaSelectShape)
_SIGS = {
    "xqa_workspace_size": [_SHAPE, ctypes.POINTER(_SZ)],
    "xqa_decode": [_P, _P, _P, _P, _P, _F, _F, _P, _SHAPE, _P, _SZ, _P],
    "xqa_plan": [_P, _SHAPE, _P, _SZ, _P],
    "xqa_attend_partial": [_P, _P, _P, _P, _P, _F, _F, _P, _SHAPE, _P, _SZ, _P],
    "xqa_combine": [_P, _F, _P, _SHAPE, _P, _SZ, _P],
    "xqa_dequant_e5m2": [_P, _SZ, _F, _P, _P, _P],
    "xqa_read_status": [_P, ctypes.POINTER(ctypes.c_int32), _P],
    "xqa_read_plan": [_P, _SHAPE, _P, _P, _P, _P, _P],
    "xqa_status_string": [ctypes.c_int],
    "xqa_decode_static_workspace": [_P, _P, _P, _P, _P, _F, _F, _P, _SHAPE, _P],
    "xqa_decode_device_scales": [_P, _P, _P, _P, _P, _P, _P, _P, _SHAPE, _P, _SZ, _P],
    "xqa_dequant_e4m3": [_P, _SZ, _F, _P, _P, _P],
    "xqa_selftest_wait_timeout": [_P, ctypes.c_uint64, _P],
    "xqa_kernels_per_call": [_SHAPE, ctypes.POINTER(ctypes.c_int32)],
    "xqa_prefill": [_P, _P, _P, _P, _P, _P, _P, _PREFILL, _P, _SZ, _P],
    "xqa_prefill_workspace_size": [_PREFILL, ctypes.POINTER(_SZ)],
    "xqa_extend": [_P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _P, _EXTEND, _P, _SZ, _P],
    "xqa_extend_workspace_size": [_EXTEND, ctypes.POINTER(_SZ)],
    "xqa_assign_pages": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _PAGES, _P, _P],
    "xqa_release_pages": [_P, _P, _P, _P, _P, _P, _P, _PAGES, _P, _P],
    "xqa_page_bounds": [_P, _P, _P, _P, _P, _ROWS, _P, _P],
    "xqa_select": [_P, _P, _P, _P, _P, _P, _SELECT, _P, _SZ, _P],
    "xqa_select_workspace_size": [_SELECT, ctypes.POINTER(_SZ)],
    "xqa_decode_selected": [_P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _SHAPE, _P, _SZ, _P],
    "xqa_append": [_P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _P, _ROWS, _P, _P],
    "xqa_gather": [_P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _P, _ROWS, _P, _P],
}


def load_library() -> ctypes.CDLL:
    """Load libxqa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()' or "
                "python paged_fp8_kv_gqa_gb300/build.py)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, argtypes in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = argtypes
            fn.restype = ctypes.c_char_p if name == "xqa_status_string" else ctypes.c_int
        _lib = lib
    return _lib


def xqa_status_string(code: int) -> str:
    return load_library().xqa_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != XQA_OK:
        raise XqaError(code, where)


def _stream_handle(stream) -> int:
    if stream is None:  # torch.cuda.current_stream() without the Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return _device_stream(stream)[1]


def _cuda(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def make_shape(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
               sm_scale: float = 0.0, max_ctas: int = 0, min_pages_per_cta: int = 0,
               merge_mode: int = 0, kv_dtype: str = "e5m2", kv_layout: str = "hnd") -> XqaShape:
    """Shape descriptor from q [B, Hq, D] (or [B, T, Hq, D] for T new tokens per
    sequence), block_tables [B, MBS] and k_cache [NB, Hkv, BS, D] (kv_layout
    "hnd") or [NB, BS, Hkv, D] ("nhd"); for kv_dtype "e2m1" [NB, Hkv, 1152]."""
    if q.dim() == 4:
        b, t_new, hq, d = q.shape
    else:
        (b, hq, d), t_new = q.shape, 1
    if kv_dtype == "e2m1":
        nb, hkv, bs = _cache_dims(k_cache, kv_dtype, kv_layout)
        d2 = 128
    elif kv_layout == "hnd":
        nb, hkv, bs, d2 = k_cache.shape
    else:
        nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or block_tables.shape[0] != b:
        raise ValueError("inconsistent q / k_cache / block_tables shapes")
    return XqaShape(int(b), int(hq), int(hkv), int(d), int(bs), int(block_tables.shape[1]),
                    int(nb), float(sm_scale), int(max_ctas), int(min_pages_per_cta),
                    int(merge_mode), KV_DTYPES[kv_dtype], KV_LAYOUTS[kv_layout], int(t_new))


def xqa_workspace_size(shape: XqaShape) -> int:
    n = _SZ(0)
    _check(load_library().xqa_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "xqa_workspace_size")
    return int(n.value)


def xqa_kernels_per_call(shape: XqaShape) -> int:
    """Kernels one xqa_decode call enqueues for this shape."""
    n = ctypes.c_int32(0)
    _check(load_library().xqa_kernels_per_call(ctypes.byref(shape), ctypes.byref(n)),
           "xqa_kernels_per_call")
    return int(n.value)


def alloc_workspace(shape: XqaShape, device=None) -> torch.Tensor:
    """A zero-filled uint8 device buffer of xqa_workspace_size bytes (256-byte
    aligned by torch). The library needs it zeroed once, before its first use;
    every call leaves it ready for the next."""
    return torch.zeros(xqa_workspace_size(shape), dtype=torch.uint8, device=device or "cuda")


@functools.lru_cache(maxsize=1024)
def _decode_fits(shape: bytes, q, k_cache, v_cache, block_tables, n_lens: int, n_out) -> bool:
    """Raises unless tensors of these shapes are what the descriptor says (n_out: elements of
    out, None if it is like q)."""
    s = XqaShape.from_buffer_copy(shape)
    if s.kv_dtype == KV_DTYPES["e2m1"]:
        page = (s.num_kv_heads, E2M1_SLICE_BYTES)
    elif s.kv_layout == KV_LAYOUTS["nhd"]:
        page = (s.block_size, s.num_kv_heads, s.head_dim)
    else:
        page = (s.num_kv_heads, s.block_size, s.head_dim)
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if c[1:] != page or c[0] < s.num_blocks:
            raise ValueError(f"{name} is {tuple(c)}, the shape descriptor says {(s.num_blocks, *page)}")
    n = s.batch * max(s.q_len, 1) * s.num_q_heads * s.head_dim
    if q[-2:] != (s.num_q_heads, s.head_dim) or q.numel() != n or n_out not in (n, None):
        raise ValueError("q or out does not match the shape descriptor")
    if len(block_tables) != 2 or block_tables[0] < s.batch or block_tables[1] != s.max_blocks_per_seq:
        raise ValueError("block_tables does not match the shape descriptor")
    if n_lens < s.batch:
        raise ValueError("context_lens has fewer entries than sequences")
    return True


def _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, workspace, shape,
                 static=False, fresh=False):
    """Pointers of a decode call's tensors, checked (static: a call without a workspace;
    fresh: out was allocated like q just now)."""
    try:  # the usual call, without a function call for each tensor
        dev = q.get_device()
        if (dev >= 0 and q.dtype is _F16 and q.is_contiguous()
                and k_cache.dtype is _U8 and k_cache.get_device() == dev and k_cache.is_contiguous()
                and v_cache.dtype is _U8 and v_cache.get_device() == dev and v_cache.is_contiguous()
                and block_tables.dtype is _I32 and block_tables.get_device() == dev
                and block_tables.is_contiguous()
                and context_lens.dtype is _I32 and context_lens.get_device() == dev
                and context_lens.is_contiguous()
                and (fresh or (out.dtype is _F16 and out.get_device() == dev and out.is_contiguous()))
                and (static or (workspace.dtype is _U8 and workspace.get_device() == dev
                                and workspace.is_contiguous()))
                and torch._C._cuda_getDevice() == dev
                and _decode_fits(bytes(shape), q.shape, k_cache.shape, v_cache.shape,
                                 block_tables.shape, context_lens.numel(),
                                 None if fresh else out.numel())):
            return (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
                    context_lens.data_ptr(), out.data_ptr(), None if static else workspace.data_ptr())
    except AttributeError:
        pass
    _on_current((q, _F16, "q"), (k_cache, _U8, "k_cache"), (v_cache, _U8, "v_cache"),  # the reason
                (block_tables, _I32, "block_tables"), (context_lens, _I32, "context_lens"),
                (out, _F16, "out"), *([] if static else [(workspace, _U8, "workspace")]))
    raise ValueError("invalid arguments")


def xqa_decode(q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale,
               out=None, workspace=None, shape: XqaShape | None = None, stream=None,
               sm_scale: float = 0.0, max_ctas: int = 0, min_pages_per_cta: int = 0,
               kv_dtype: str = "e5m2", kv_layout: str = "hnd"):
    """One decode step. Tensors: q fp16 [B,Hq,D]; k/v_cache uint8 FP8 codes
    [NB,Hkv,16,D] (or [NB,16,Hkv,D] for kv_layout "nhd"), for kv_dtype "e2m1"
    4-bit slices [NB,Hkv,1152]; block_tables int32 [B,MBS]; context_lens int32
    [B]. k_scale / v_scale are floats, or float32 CUDA tensors of one element
    (read on the device: xqa_decode_device_scales). Returns ``out`` fp16 [B,Hq,D]."""
    if shape is None:
        shape = make_shape(q, k_cache, block_tables, sm_scale, max_ctas, min_pages_per_cta,
                           kv_dtype=kv_dtype, kv_layout=kv_layout)
    fresh = out is None
    if fresh and workspace is not None and stream is None:
        out = torch.empty_like(q)
    elif out is None or workspace is None:
        with _allocating(stream):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = alloc_workspace(shape, q.device)
    a = _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, workspace, shape,
                     fresh=fresh)
    lib = load_library()
    # the tensors are on the current device
    handle = (torch._C._cuda_getCurrentRawStream(q.get_device()) if stream is None
              else _stream_handle(stream))
    if not (type(k_scale) is type(v_scale) is float) and (
            isinstance(k_scale, torch.Tensor) or isinstance(v_scale, torch.Tensor)):
        ks, vs = (_on(x, torch.float32, q.get_device(), name)
                  for x, name in ((k_scale, "k_scale"), (v_scale, "v_scale")))
        _check(lib.xqa_decode_device_scales(a[0], a[1], a[2], a[3], a[4], ks, vs, a[5],
                                            ctypes.byref(shape), a[6], workspace.numel(),
                                            handle), "xqa_decode_device_scales")
        return out
    code = lib.xqa_decode(a[0], a[1], a[2], a[3], a[4], float(k_scale), float(v_scale), a[5],
                          ctypes.byref(shape), a[6], workspace.numel(), handle)
    if code:
        raise XqaError(code, "xqa_decode")
    return out


def _on_current(*named) -> list:
    """Pointers of (tensor, dtype, name) on the current device."""
    for t, dtype, name in named:  # CPU tensors before CUDA is asked
        _cuda(t, dtype, name)
    dev = torch.cuda.current_device()
    return [_on(t, dtype, dev, name) for t, dtype, name in named]


def xqa_plan(context_lens, workspace, shape: XqaShape, stream=None) -> None:
    lens, ws = _on_current((context_lens, _I32, "context_lens"), (workspace, _U8, "workspace"))
    if context_lens.numel() < shape.batch:
        raise ValueError("context_lens has fewer entries than sequences")
    _check(load_library().xqa_plan(lens, ctypes.byref(shape), ws, workspace.numel(),
                                   _stream_handle(stream)), "xqa_plan")


def xqa_attend_partial(q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, out,
                       workspace, shape: XqaShape, stream=None) -> None:
    a = _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, workspace, shape)
    _check(load_library().xqa_attend_partial(a[0], a[1], a[2], a[3], a[4], float(k_scale),
                                             float(v_scale), a[5], ctypes.byref(shape), a[6],
                                             workspace.numel(), _stream_handle(stream)),
           "xqa_attend_partial")


def xqa_combine(context_lens, v_scale, out, workspace, shape: XqaShape, stream=None) -> None:
    o, lens, ws = _on_current((out, _F16, "out"), (context_lens, _I32, "context_lens"),
                              (workspace, _U8, "workspace"))
    if out.numel() != shape.batch * max(shape.q_len, 1) * shape.num_q_heads * shape.head_dim:
        raise ValueError("out does not match the shape descriptor")
    _check(load_library().xqa_combine(lens, float(v_scale), o, ctypes.byref(shape), ws,
                                      workspace.numel(), _stream_handle(stream)), "xqa_combine")


def _dequant(fn_name, codes, scale, with_f32, stream):
    n = codes.numel()
    out16 = torch.empty(n, dtype=torch.int16, device=codes.device)
    out32 = torch.empty(n, dtype=torch.float32, device=codes.device) if with_f32 else None
    _check(getattr(load_library(), fn_name)(
        _cuda(codes, torch.uint8, "codes"), n, float(scale), out16.data_ptr(),
        out32.data_ptr() if out32 is not None else None, _stream_handle(stream)), fn_name)
    return out16, out32


def xqa_dequant_e5m2(codes: torch.Tensor, scale: float = 1.0, with_f32: bool = True, stream=None):
    """Exact dequantisation: returns (fp16 bit patterns as int16 tensor, fp32 scaled or None)."""
    return _dequant("xqa_dequant_e5m2", codes, scale, with_f32, stream)


def xqa_dequant_e4m3(codes: torch.Tensor, scale: float = 1.0, with_f32: bool = True, stream=None):
    """Exact E4M3 dequantisation: (fp16 bit patterns as int16 tensor, fp32 scaled or None)."""
    return _dequant("xqa_dequant_e4m3", codes, scale, with_f32, stream)


_NO_CONTEXT = contextlib.nullcontext()


def _allocating(stream):
    """Context in which the binding allocates what a call on ``stream`` writes: the
    memory (and the zero fill of a workspace) belongs to that stream."""
    return torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream) else _NO_CONTEXT


def _device_stream(stream):
    """(current device, handle of ``stream`` or of its current stream). The
    library works on the current device: the stream must be there, and every
    tensor (checked where its pointer is taken)."""
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if getattr(stream, "device_index", dev) != dev:  # (any object with a cuda_stream will do)
        raise ValueError("the stream belongs to another device than the current one")
    return dev, int(stream.cuda_stream)


def _on(t: torch.Tensor, dtype, dev: int, name: str) -> int:
    """Pointer of a contiguous tensor of ``dtype`` on device ``dev``."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    _cuda(t, dtype, name)  # raises with the reason, if it is not the device
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _heads(t: torch.Tensor, name: str, dtype=None):
    """(row stride, head stride) of a [rows, heads, 128] CUDA view whose last
    dim is contiguous (strides of dims of size 1 play no part)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in ROW_DTYPES or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must have dtype {dtype or 'float16 or bfloat16'}, got {t.dtype}")
    return _head_strides(t.shape, t.stride(), name)


def _head_strides(shape, stride, name: str):
    if len(shape) != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim], got {tuple(shape)}")
    n, h, d = shape
    if n == 0 or h == 0:
        return h * d, d
    rs, hs, es = stride
    if h == 1:
        hs = d
    if n == 1:
        rs = h * d
    if (es != 1 and d > 1) or rs <= 0 or hs <= 0:
        raise ValueError(f"{name}: the last dim must be contiguous and no stride may be 0")
    return rs, hs


def _cache_dims(cache: torch.Tensor, kv_dtype: str, kv_layout: str):
    """(num_blocks, num_kv_heads, block_size) of a cache tensor."""
    return _cache_shape(cache.shape, kv_dtype, kv_layout)


def _cache_shape(shape, kv_dtype: str, kv_layout: str):
    if kv_dtype == "e2m1":
        if len(shape) != 3 or shape[2] != E2M1_SLICE_BYTES or kv_layout != "hnd":
            raise ValueError("an e2m1 cache is [num_blocks, num_kv_heads, 1152], kv_layout 'hnd'")
        return shape[0], shape[1], 16
    if len(shape) != 4:
        raise ValueError("an FP8 cache has four dims")
    nb, a, b, d = shape
    if d != 128:
        raise ValueError("head_dim must be 128")
    return (nb, a, b) if kv_layout == "hnd" else (nb, b, a)


def _scale_arg(s, dev: int, name: str):
    """(value, pointer) of a scale: a float, or a CUDA tensor of one element."""
    if not isinstance(s, torch.Tensor):
        return float(s), None
    if s.numel() != 1:
        raise ValueError(f"{name} must have one element")
    return 0.0, _on(s, torch.float32, dev, name)


@functools.lru_cache(maxsize=1024)
def _rows_descriptor(k_shape, k_stride, v_shape, v_stride, kc_shape, vc_shape, bt_shape, n_lens,
                     n_cu, dtype, kv_dtype, kv_layout) -> XqaRows:
    """The descriptor of calls with tensors of these shapes and strides, checked."""
    krs, khs = _head_strides(k_shape, k_stride, "k")
    vrs, vhs = _head_strides(v_shape, v_stride, "v")
    nb, hkv, bs = _cache_shape(kc_shape, kv_dtype, kv_layout)
    n, h, d = k_shape
    if (v_shape != k_shape or vc_shape != kc_shape or h != hkv or d != 128
            or len(bt_shape) != 2 or bt_shape[0] != n_lens or n_cu != n_lens + 1):
        raise ValueError("inconsistent rows / cache / block_tables / cu_seqlens shapes")
    if dtype not in ROW_DTYPES:
        raise ValueError(f"k must have dtype float16 or bfloat16, got {dtype}")
    return XqaRows(n_lens, hkv, 128, bs, bt_shape[1], nb, n, KV_DTYPES[kv_dtype],
                   KV_LAYOUTS[kv_layout], ROW_DTYPES[dtype], krs, khs, vrs, vhs)


def _refuse_rows(k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens, stream):
    """Raises with the first reason to refuse a call of _move_rows."""
    _heads(k, "k")  # CPU tensors before CUDA is asked
    _heads(v, "v", k.dtype)
    dev, _ = _device_stream(stream)
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"k and v must be on the current device, cuda:{dev}")
    for x, dtype, name in ((k_cache, _U8, "k_cache"), (v_cache, _U8, "v_cache"),
                           (cu_seqlens, _I32, "cu_seqlens"), (block_tables, _I32, "block_tables"),
                           (context_lens, _I32, "context_lens")):
        _on(x, dtype, dev, name)
    raise ValueError("invalid arguments")


def _move_rows(fn_name, k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens, k_scale,
               v_scale, kv_dtype, kv_layout, status, stream):
    rows = None
    try:  # the usual call, without a function call for each tensor
        dev, dtype = k.get_device(), k.dtype
        if (dev >= 0 and v.dtype is dtype and v.get_device() == dev
                and k_cache.dtype is _U8 and k_cache.get_device() == dev and k_cache.is_contiguous()
                and v_cache.dtype is _U8 and v_cache.get_device() == dev and v_cache.is_contiguous()
                and cu_seqlens.dtype is _I32 and cu_seqlens.get_device() == dev
                and cu_seqlens.is_contiguous()
                and block_tables.dtype is _I32 and block_tables.get_device() == dev
                and block_tables.is_contiguous()
                and context_lens.dtype is _I32 and context_lens.get_device() == dev
                and context_lens.is_contiguous() and torch._C._cuda_getDevice() == dev):
            rows = _rows_descriptor(k.shape, k.stride(), v.shape, v.stride(), k_cache.shape,
                                    v_cache.shape, block_tables.shape, context_lens.numel(),
                                    cu_seqlens.numel(), dtype, kv_dtype, kv_layout)
    except AttributeError:
        pass
    if rows is None:
        _refuse_rows(k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens, stream)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    ks, ksp = (k_scale, None) if type(k_scale) is float else _scale_arg(k_scale, dev, "k_scale")
    vs, vsp = (v_scale, None) if type(v_scale) is float else _scale_arg(v_scale, dev, "v_scale")
    kp, vp, kc, vc = k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    if fn_name == "xqa_append":
        fn = load_library().xqa_append
    else:
        fn, kp, vp, kc, vc = load_library().xqa_gather, kc, vc, kp, vp
    code = fn(kp, vp, cu_seqlens.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), ks, vs,
              ksp, vsp, kc, vc, ctypes.byref(rows),
              None if status is None else _on(status, _I32, dev, "status"), handle)
    if code:
        raise XqaError(code, fn_name)


def xqa_append(k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale,
               kv_dtype: str = "e5m2", kv_layout: str = "hnd", status=None, stream=None) -> None:
    """Write new tokens' keys and values into the paged cache. k, v: fp16 or bf16
    [rows, Hkv, 128] (views with strides are fine), packed by sequence through
    cu_seqlens int32 [B+1]; context_lens int32 [B] counts the new tokens, which
    go to each sequence's last positions. k_cache / v_cache: uint8, [NB, Hkv, 16,
    128] ("hnd"), [NB, 16, Hkv, 128] ("nhd") or, for kv_dtype "e2m1", [NB, Hkv,
    1152]. Scales are floats, or float32 CUDA tensors of one element. ``status``
    (int32 CUDA tensor, optional) receives the first device-side error."""
    _move_rows("xqa_append", k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens,
               k_scale, v_scale, kv_dtype, kv_layout, status, stream)


def xqa_gather(k_cache, v_cache, block_tables, context_lens, cu_seqlens, num_rows: int, k_scale,
               v_scale, dtype=torch.float16, kv_dtype: str = "e5m2", kv_layout: str = "hnd",
               k=None, v=None, status=None, stream=None):
    """Read cached tokens back as packed rows of ``dtype``: sequence b's rows
    cu_seqlens[b] .. cu_seqlens[b+1]-1 receive its last tokens (all of them when
    there are context_lens[b] rows). Returns (k, v), [num_rows, Hkv, 128]; pass
    ``k`` and ``v`` to write into existing tensors or views (rows behind the last
    sequence are left as they are)."""
    if (k is None) != (v is None):
        raise ValueError("pass both k and v, or neither")
    if k is None:
        hkv = _cache_dims(k_cache, kv_dtype, kv_layout)[1]
        with _allocating(stream) if stream is not None else _NO_CONTEXT:
            k = torch.empty((int(num_rows), hkv, 128), dtype=dtype, device=k_cache.device)
            v = torch.empty_like(k)
    elif k.shape[0] != num_rows:
        raise ValueError("k and v must have num_rows rows")
    _move_rows("xqa_gather", k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens,
               k_scale, v_scale, kv_dtype, kv_layout, status, stream)
    return k, v


def make_prefill_shape(q, k, v, cu_seqlens_q, causal: bool = True, sm_scale: float = 0.0,
                       max_ctas: int = 0, out=None) -> XqaPrefillShape:
    """Shape descriptor of xqa_prefill from q [total_q, Hq, 128], k and v
    [total_k, Hkv, 128] (fp16 or bf16; views whose last dim is contiguous are
    fine) and cu_seqlens_q [B+1]. It holds for every call with tensors of these
    shapes, types and strides (out: contiguous unless given)."""
    side = _prefill_strides(q, k, v)
    orow, oh = (0, 0) if out is None else _heads(out, "out", q.dtype)
    return XqaPrefillShape(cu_seqlens_q.numel() - 1, q.shape[1], k.shape[1], q.shape[2],
                           q.shape[0], k.shape[0], ROW_DTYPES[q.dtype], int(bool(causal)),
                           float(sm_scale), int(max_ctas), *side, orow, oh)


def _prefill_strides(q, k, v):
    side = _heads(q, "q") + _heads(k, "k", q.dtype) + _heads(v, "v", q.dtype)
    if k.shape != v.shape or k.shape[2] != q.shape[2]:
        raise ValueError("inconsistent q / k / v shapes")
    return side


@functools.lru_cache(maxsize=1024)
def _prefill_fields(q_shape, q_stride, k_shape, k_stride, v_shape, v_stride, dtype) -> tuple:
    """(what a descriptor for tensors of these shapes and strides holds from num_q_heads to
    dtype, and as strides; its strides of a contiguous out, written out or 0)."""
    side = (_head_strides(q_shape, q_stride, "q") + _head_strides(k_shape, k_stride, "k")
            + _head_strides(v_shape, v_stride, "v"))
    if k_shape != v_shape or k_shape[2] != q_shape[2] or dtype not in ROW_DTYPES:
        raise ValueError("inconsistent q / k / v shapes")
    rs, hs = q_shape[1] * q_shape[2], q_shape[2]
    s = bytes(XqaPrefillShape(0, q_shape[1], k_shape[1], q_shape[2], q_shape[0], k_shape[0],
                              ROW_DTYPES[dtype], 0, 0.0, 0, *side, 0, 0))
    outs = frozenset(bytes(XqaPrefillShape(out_row_stride=a, out_head_stride=b))[_OUT_AT:]
                     for a in (0, rs) for b in (0, hs))
    return s[_DIMS_AT:_CAUSAL_AT], s[_STRIDES_AT:_OUT_AT], outs


def xqa_prefill_workspace_size(shape: XqaPrefillShape) -> int:
    n = _SZ(0)
    _check(load_library().xqa_prefill_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "xqa_prefill_workspace_size")
    return int(n.value)


def alloc_prefill_workspace(shape: XqaPrefillShape, device=None) -> torch.Tensor:
    """A zero-filled uint8 device buffer of xqa_prefill_workspace_size bytes;
    every call leaves it ready for the next."""
    return torch.zeros(xqa_prefill_workspace_size(shape), dtype=torch.uint8,
                       device=device or "cuda")


def _refuse_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k, stream):
    """Raises with the first reason to refuse a call of xqa_prefill."""
    _prefill_strides(q, k, v)  # CPU tensors before CUDA is asked
    dev, _ = _device_stream(stream)
    for x in (q, k, v):
        if x.get_device() != dev:
            raise ValueError(f"q, k, v and out must be on the current device, cuda:{dev}")
    _on(cu_seqlens_q, _I32, dev, "cu_seqlens_q")
    _on(cu_seqlens_k, _I32, dev, "cu_seqlens_k")
    raise ValueError("invalid arguments")


def xqa_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k=None, out=None, lse=None, workspace=None,
                shape: XqaPrefillShape | None = None, stream=None, causal: bool = True,
                sm_scale: float = 0.0, max_ctas: int = 0):
    """Attention of whole prompts, packed by sequence: q fp16 or bf16 [total_q,
    Hq, 128], k and v [total_k, Hkv, 128], cu_seqlens_q / cu_seqlens_k int32
    [B+1] (keys default to the queries' offsets). With ``causal`` the last query
    of a sequence sees all its keys and each one before it one key less. ``lse``
    (fp32 [total_q, Hq], optional) receives the log-sum-exp. Returns ``out``;
    rows that see nothing are zero, rows behind the last sequence are not
    written. Errors that only the device sees (bad offsets, a wait that ran out)
    are in the workspace: pass one and call xqa_read_status on it to learn of
    them. Without ``workspace`` the call allocates one and drops it, status
    included."""
    if shape is None:
        shape = make_prefill_shape(q, k, v, cu_seqlens_q, causal, sm_scale, max_ctas, out)
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens_q
    outs = None
    try:  # the usual call, without a function call for each tensor
        dev, dtype = q.get_device(), q.dtype
        if (dev >= 0 and k.dtype is dtype and k.get_device() == dev
                and v.dtype is dtype and v.get_device() == dev
                and cu_seqlens_q.dtype is _I32 and cu_seqlens_q.get_device() == dev
                and cu_seqlens_q.is_contiguous()
                and cu_seqlens_k.dtype is _I32 and cu_seqlens_k.get_device() == dev
                and cu_seqlens_k.is_contiguous() and torch._C._cuda_getDevice() == dev):
            dims, strides, outs = _prefill_fields(q.shape, q.stride(), k.shape, k.stride(), v.shape,
                                                  v.stride(), dtype)
    except AttributeError:
        pass
    if outs is None:
        _refuse_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k, stream)
    held = bytes(shape)
    if held[_DIMS_AT:_CAUSAL_AT] != dims or held[_STRIDES_AT:_OUT_AT] != strides:
        raise ValueError("q, k, v do not match the shape descriptor")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    if out is None:
        if held[_OUT_AT:] not in outs:
            raise ValueError("the shape descriptor names strides of out: pass out")
        with _allocating(stream) if stream is not None else _NO_CONTEXT:
            out = torch.empty(q.shape, dtype=dtype, device=q.device)
    elif out.shape != q.shape or _heads(out, "out", dtype) != (
            shape.out_row_stride or shape.num_q_heads * 128, shape.out_head_stride or 128):
        raise ValueError("out does not match q or the shape descriptor")
    elif out.get_device() != dev:
        raise ValueError(f"q, k, v and out must be on the current device, cuda:{dev}")
    if workspace is None:
        with _allocating(stream):
            workspace = alloc_prefill_workspace(shape, q.device)
    n = shape.batch + 1
    if cu_seqlens_q.numel() != n or cu_seqlens_k.numel() != n:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have batch + 1 entries")
    lp = None
    if lse is not None:
        lp = _on(lse, torch.float32, dev, "lse")
        if lse.shape != q.shape[:2]:
            raise ValueError("lse must be [total_q, num_q_heads]")
    code = load_library().xqa_prefill(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
        out.data_ptr(), lp, ctypes.byref(shape), _on(workspace, _U8, dev, "workspace"),
        workspace.numel(), handle)
    if code:
        raise XqaError(code, "xqa_prefill")
    return out


def make_extend_shape(q, k_cache, block_tables, causal: bool = True, sm_scale: float = 0.0,
                      max_ctas: int = 0, kv_dtype: str = "e5m2", kv_layout: str = "hnd",
                      out=None) -> XqaExtendShape:
    """Shape descriptor of xqa_extend from q [total_q, Hq, 128] (fp16 or bf16; a view whose
    last dim is contiguous is fine), k_cache as for xqa_decode and block_tables [B, MBS].
    It holds for every call with tensors of these shapes, types and strides (out:
    contiguous unless given)."""
    qs = _heads(q, "q")
    orow, oh = (0, 0) if out is None else _heads(out, "out", q.dtype)
    nb, hkv, bs = _cache_dims(k_cache, kv_dtype, kv_layout)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq]")
    return XqaExtendShape(block_tables.shape[0], q.shape[1], hkv, q.shape[2], bs,
                          block_tables.shape[1], nb, q.shape[0], ROW_DTYPES[q.dtype],
                          KV_DTYPES[kv_dtype], KV_LAYOUTS[kv_layout], int(bool(causal)),
                          float(sm_scale), int(max_ctas), *qs, orow, oh)


def xqa_extend_workspace_size(shape: XqaExtendShape) -> int:
    n = _SZ(0)
    _check(load_library().xqa_extend_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "xqa_extend_workspace_size")
    return int(n.value)


def alloc_extend_workspace(shape: XqaExtendShape, device=None) -> torch.Tensor:
    """A zero-filled uint8 device buffer of xqa_extend_workspace_size bytes; every call
    leaves it ready for the next."""
    return torch.zeros(xqa_extend_workspace_size(shape), dtype=torch.uint8, device=device or "cuda")


@functools.lru_cache(maxsize=1024)
def _extend_fits(shape: bytes, q_shape, q_stride, dtype, k_cache, v_cache, block_tables,
                 n_lens: int, n_cu: int) -> bool:
    """Raises unless tensors of these shapes are what the descriptor says; whether a
    contiguous out is what it says too."""
    s = XqaExtendShape.from_buffer_copy(shape)
    names = {v: k for k, v in KV_DTYPES.items()}, {v: k for k, v in KV_LAYOUTS.items()}
    rs, hs = _head_strides(q_shape, q_stride, "q")
    if (dtype not in ROW_DTYPES or ROW_DTYPES[dtype] != s.dtype
            or tuple(q_shape) != (s.total_q, s.num_q_heads, s.head_dim)
            or rs != (s.q_row_stride or s.num_q_heads * 128) or hs != (s.q_head_stride or 128)):
        raise ValueError("q does not match the shape descriptor")
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        nb, hkv, bs = _cache_shape(c, names[0][s.kv_dtype], names[1][s.kv_layout])
        if (hkv, bs) != (s.num_kv_heads, s.block_size) or nb < s.num_blocks or c != k_cache:
            raise ValueError(f"{name} does not match the shape descriptor")
    if tuple(block_tables) != (s.batch, s.max_blocks_per_seq):
        raise ValueError("block_tables does not match the shape descriptor")
    if n_lens != s.batch or n_cu != s.batch + 1:
        raise ValueError("context_lens must have batch entries, cu_seqlens batch + 1")
    return s.out_row_stride in (0, s.num_q_heads * 128) and s.out_head_stride in (0, 128)


def xqa_extend(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, k_scale, v_scale,
               out=None, lse=None, workspace=None, shape: XqaExtendShape | None = None, stream=None,
               causal: bool = True, sm_scale: float = 0.0, max_ctas: int = 0,
               kv_dtype: str = "e5m2", kv_layout: str = "hnd"):
    """Attention of chunks of new tokens over the paged cache. q: fp16 or bf16 [total_q, Hq,
    128], packed by sequence through cu_seqlens int32 [B+1]; the chunk's own keys and values
    are in the cache already (xqa_append), and context_lens int32 [B] counts them. Query i
    of a sequence's n sees its tokens 0 .. context_len - n + i (all of them without
    ``causal``). Caches, block_tables and scales as for xqa_decode. ``lse`` (fp32 [total_q,
    Hq], optional) receives the log-sum-exp. Returns ``out``; rows that see nothing are
    zero, rows behind the last sequence are not written. Errors that only the device sees
    are in the workspace (xqa_read_status); without ``workspace`` the call allocates one
    and drops it, status included."""
    if shape is None:
        shape = make_extend_shape(q, k_cache, block_tables, causal, sm_scale, max_ctas, kv_dtype,
                                  kv_layout, out)
    plain_out = None
    try:  # the usual call, without a function call for each tensor
        dev, dtype = q.get_device(), q.dtype
        if (dev >= 0 and k_cache.dtype is _U8 and k_cache.get_device() == dev and k_cache.is_contiguous()
                and v_cache.dtype is _U8 and v_cache.get_device() == dev and v_cache.is_contiguous()
                and block_tables.dtype is _I32 and block_tables.get_device() == dev
                and block_tables.is_contiguous()
                and context_lens.dtype is _I32 and context_lens.get_device() == dev
                and context_lens.is_contiguous()
                and cu_seqlens.dtype is _I32 and cu_seqlens.get_device() == dev
                and cu_seqlens.is_contiguous() and torch._C._cuda_getDevice() == dev):
            plain_out = _extend_fits(bytes(shape), q.shape, q.stride(), dtype, k_cache.shape,
                                     v_cache.shape, block_tables.shape, context_lens.numel(),
                                     cu_seqlens.numel())
    except AttributeError:
        pass
    if plain_out is None:
        _heads(q, "q")
        _on_current((k_cache, _U8, "k_cache"), (v_cache, _U8, "v_cache"),
                    (block_tables, _I32, "block_tables"), (context_lens, _I32, "context_lens"),
                    (cu_seqlens, _I32, "cu_seqlens"))
        raise ValueError("q must be on the current device")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    if out is None:
        if not plain_out:
            raise ValueError("the shape descriptor names strides of out: pass out")
        out = _like(q, q.shape, stream)
    elif out.shape != q.shape or _heads(out, "out", dtype) != (
            shape.out_row_stride or shape.num_q_heads * 128, shape.out_head_stride or 128):
        raise ValueError("out does not match q or the shape descriptor")
    elif out.get_device() != dev:
        raise ValueError(f"q and out must be on the current device, cuda:{dev}")
    if workspace is None:
        with _allocating(stream):
            workspace = alloc_extend_workspace(shape, q.device)
    lp = None
    if lse is not None:
        lp = _on(lse, torch.float32, dev, "lse")
        if lse.shape != q.shape[:2]:
            raise ValueError("lse must be [total_q, num_q_heads]")
    ks, ksp = (k_scale, None) if type(k_scale) is float else _scale_arg(k_scale, dev, "k_scale")
    vs, vsp = (v_scale, None) if type(v_scale) is float else _scale_arg(v_scale, dev, "v_scale")
    code = load_library().xqa_extend(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), cu_seqlens.data_ptr(), ks, vs, ksp, vsp, out.data_ptr(), lp,
        ctypes.byref(shape), _on(workspace, _U8, dev, "workspace"), workspace.numel(), handle)
    if code:
        raise XqaError(code, "xqa_extend")
    return out


_BOOL = torch.bool


@functools.lru_cache(maxsize=1024)
def _pages_descriptor(n_lens: int, bt_shape, n_free: int, n_first: int, num_rows: int, *single) -> XqaPages:
    """The descriptor of calls with tensors of these sizes, checked (n_first: entries of
    new_tokens or done; single: sizes that have to be 1, B or B + 1 with what they have to be)."""
    if len(bt_shape) != 2 or bt_shape[0] != n_lens or n_first != n_lens:
        raise ValueError("inconsistent context_lens / block_tables / new_tokens or done")
    for have, want in zip(single[::2], single[1::2]):
        if have != want:
            raise ValueError(f"a tensor has {have} entries where {want} are needed")
    return XqaPages(n_lens, 16, bt_shape[1], n_free, num_rows)


def _like(t: torch.Tensor, shape, stream) -> torch.Tensor:
    """An uninitialised tensor of t's type and device that a call on ``stream`` writes."""
    if stream is None:
        return torch.empty(shape, dtype=t.dtype, device=t.device)
    with _allocating(stream):
        return torch.empty(shape, dtype=t.dtype, device=t.device)


def _all_i32(dev: int, *tensors) -> bool:
    for t in tensors:
        if not (t.dtype is _I32 and t.get_device() == dev and t.is_contiguous()):
            return False
    return True


def xqa_assign_pages(new_tokens, context_lens, block_tables, free_pages, num_free, num_rows: int,
                     new_lens=None, new_free=None, cu_seqlens=None, slots=None, positions=None,
                     status=None, stream=None):
    """Give a step's new tokens their pages. new_tokens, context_lens: int32 [B];
    block_tables: int32 [B, MBS], written where a sequence gets a page; free_pages: int32
    [NB], of which the first ``num_free`` (int32 CUDA tensor of one element) are a stack of
    free pages. context_lens and num_free become what they are after the step, or stay if
    ``new_lens`` and ``new_free`` are passed. Returns (cu_seqlens [B+1], slots [num_rows],
    positions [num_rows]), int32: the new tokens' offsets, and for each the slot page * 16 +
    position % 16 and the position (-1 in rows behind the last). A sequence that cannot be
    served gains nothing; ``status`` (int32 CUDA tensor, optional) receives the first error
    of that kind."""
    new_lens = context_lens if new_lens is None else new_lens
    new_free = num_free if new_free is None else new_free
    pages = None
    try:  # the usual call, without a function call for each tensor
        dev = context_lens.get_device()
        if dev >= 0 and torch._C._cuda_getDevice() == dev and _all_i32(
                dev, new_tokens, context_lens, block_tables, free_pages, num_free, new_lens, new_free):
            n, num_rows = context_lens.numel(), int(num_rows)
            if num_rows < 0:
                raise ValueError("num_rows must not be negative")
            if cu_seqlens is None:
                cu_seqlens = _like(context_lens, n + 1, stream)
            if slots is None:
                slots = _like(context_lens, num_rows, stream)
            if positions is None:
                positions = _like(context_lens, num_rows, stream)
            if _all_i32(dev, cu_seqlens, slots, positions):
                pages = _pages_descriptor(n, block_tables.shape, free_pages.numel(), new_tokens.numel(),
                                          num_rows, num_free.numel(), 1, new_free.numel(), 1,
                                          new_lens.numel(), n, cu_seqlens.numel(), n + 1,
                                          slots.numel(), num_rows, positions.numel(), num_rows)
    except AttributeError:
        pass
    if pages is None:
        _on_current(*[(t, _I32, name) for t, name in (
            (new_tokens, "new_tokens"), (context_lens, "context_lens"), (block_tables, "block_tables"),
            (free_pages, "free_pages"), (num_free, "num_free"), (new_lens, "new_lens"),
            (new_free, "new_free"), (cu_seqlens, "cu_seqlens"), (slots, "slots"),
            (positions, "positions")) if t is not None or name not in ("cu_seqlens", "slots", "positions")])
        raise ValueError("invalid arguments")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    code = load_library().xqa_assign_pages(
        new_tokens.data_ptr(), context_lens.data_ptr(), block_tables.data_ptr(), free_pages.data_ptr(),
        num_free.data_ptr(), new_lens.data_ptr(), new_free.data_ptr(), cu_seqlens.data_ptr(),
        slots.data_ptr(), positions.data_ptr(), ctypes.byref(pages),
        None if status is None else _on(status, _I32, dev, "status"), handle)
    if code:
        raise XqaError(code, "xqa_assign_pages")
    return cu_seqlens, slots, positions


def xqa_release_pages(done, context_lens, block_tables, free_pages, num_free, new_lens=None,
                      new_free=None, status=None, stream=None) -> None:
    """Put the pages of ended sequences back: those of every b with ``done[b]`` (bool or uint8
    [B]) go onto the stack free_pages[:num_free], and its length becomes 0. Other arguments
    as for xqa_assign_pages."""
    new_lens = context_lens if new_lens is None else new_lens
    new_free = num_free if new_free is None else new_free
    pages = None
    try:  # the usual call, without a function call for each tensor
        dev = context_lens.get_device()
        if (dev >= 0 and torch._C._cuda_getDevice() == dev
                and (done.dtype is _BOOL or done.dtype is _U8) and done.get_device() == dev
                and done.is_contiguous()
                and _all_i32(dev, context_lens, block_tables, free_pages, num_free, new_lens, new_free)):
            n = context_lens.numel()
            pages = _pages_descriptor(n, block_tables.shape, free_pages.numel(), done.numel(), 0,
                                      num_free.numel(), 1, new_free.numel(), 1, new_lens.numel(), n)
    except AttributeError:
        pass
    if pages is None:
        _on_current(*[(t, _I32, name) for t, name in (
            (context_lens, "context_lens"), (block_tables, "block_tables"), (free_pages, "free_pages"),
            (num_free, "num_free"), (new_lens, "new_lens"), (new_free, "new_free"))])
        _on_current((done, _U8, "done"))
        raise ValueError("invalid arguments")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    code = load_library().xqa_release_pages(
        done.data_ptr(), context_lens.data_ptr(), block_tables.data_ptr(), free_pages.data_ptr(),
        num_free.data_ptr(), new_lens.data_ptr(), new_free.data_ptr(), ctypes.byref(pages),
        None if status is None else _on(status, _I32, dev, "status"), handle)
    if code:
        raise XqaError(code, "xqa_release_pages")


def alloc_bounds(k_cache, kv_dtype: str = "e5m2", kv_layout: str = "hnd") -> torch.Tensor:
    """A zero-filled uint8 buffer [num_blocks, Hkv, 272] for the bounds of k_cache's pages."""
    nb, hkv, _ = _cache_dims(k_cache, kv_dtype, kv_layout)
    return torch.zeros((nb, hkv, BOUNDS_BYTES), dtype=_U8, device=k_cache.device)


@functools.lru_cache(maxsize=1024)
def _bounds_descriptor(kc_shape, bounds_shape, bt_shape, n_lens: int, n_cu: int, num_rows: int,
                       kv_dtype, kv_layout) -> XqaRows:
    nb, hkv, bs = _cache_shape(kc_shape, kv_dtype, kv_layout)
    if (tuple(bounds_shape) != (nb, hkv, BOUNDS_BYTES) or len(bt_shape) != 2 or bt_shape[0] != n_lens
            or n_cu != n_lens + 1):
        raise ValueError("inconsistent k_cache / bounds / block_tables / cu_seqlens shapes")
    return XqaRows(n_lens, hkv, 128, bs, bt_shape[1], nb, num_rows, KV_DTYPES[kv_dtype],
                   KV_LAYOUTS[kv_layout])


def xqa_page_bounds(k_cache, block_tables, context_lens, cu_seqlens, num_rows: int, bounds,
                    kv_dtype: str = "e5m2", kv_layout: str = "hnd", status=None, stream=None) -> None:
    """Bring ``bounds`` (uint8 [NB, Hkv, 272], see alloc_bounds) up to date for the pages that a
    step's new tokens touched: after xqa_append, with its cu_seqlens and context_lens.
    ``num_rows``: rows of that call (cu_seqlens[-1] or more)."""
    rows = None
    try:  # the usual call, without a function call for each tensor
        dev = k_cache.get_device()
        if (dev >= 0 and torch._C._cuda_getDevice() == dev and k_cache.dtype is _U8
                and k_cache.is_contiguous() and bounds.dtype is _U8 and bounds.get_device() == dev
                and bounds.is_contiguous() and _all_i32(dev, block_tables, context_lens, cu_seqlens)):
            rows = _bounds_descriptor(k_cache.shape, bounds.shape, block_tables.shape,
                                      context_lens.numel(), cu_seqlens.numel(), int(num_rows), kv_dtype,
                                      kv_layout)
    except AttributeError:
        pass
    if rows is None:
        _on_current((k_cache, _U8, "k_cache"), (bounds, _U8, "bounds"), (block_tables, _I32, "block_tables"),
                    (context_lens, _I32, "context_lens"), (cu_seqlens, _I32, "cu_seqlens"))
        raise ValueError("invalid arguments")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    code = load_library().xqa_page_bounds(
        k_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), cu_seqlens.data_ptr(),
        bounds.data_ptr(), ctypes.byref(rows), None if status is None else _on(status, _I32, dev, "status"),
        handle)
    if code:
        raise XqaError(code, "xqa_page_bounds")


def make_select_shape(q, bounds, block_tables, max_pages: int, first_pages: int = 1,
                      last_pages: int = 1, max_ctas: int = 0) -> XqaSelectShape:
    """Shape descriptor of xqa_select from q [B, Hq, 128], bounds [NB, Hkv, 272] and
    block_tables [B, MBS]. It holds for every call with tensors of these shapes."""
    if q.dim() != 3 or bounds.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("q must be [B, Hq, 128], bounds [NB, Hkv, 272], block_tables [B, MBS]")
    if block_tables.shape[0] != q.shape[0] or bounds.shape[2] != BOUNDS_BYTES:
        raise ValueError("inconsistent q / bounds / block_tables shapes")
    return XqaSelectShape(q.shape[0], q.shape[1], bounds.shape[1], q.shape[2], 16,
                          block_tables.shape[1], bounds.shape[0], int(max_pages), int(first_pages),
                          int(last_pages), int(max_ctas))


def xqa_select_workspace_size(shape: XqaSelectShape) -> int:
    n = _SZ(0)
    _check(load_library().xqa_select_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "xqa_select_workspace_size")
    return int(n.value)


def alloc_select_workspace(shape: XqaSelectShape, device=None) -> torch.Tensor:
    """A zero-filled uint8 device buffer of xqa_select_workspace_size bytes; every call
    leaves it ready for the next."""
    return torch.zeros(xqa_select_workspace_size(shape), dtype=torch.uint8, device=device or "cuda")


@functools.lru_cache(maxsize=1024)
def _select_fits(shape: bytes, q, bounds, block_tables, n_lens: int, selected, selected_lens) -> bool:
    """Raises unless tensors of these shapes are what the descriptor says."""
    s = XqaSelectShape.from_buffer_copy(shape)
    if (tuple(q) != (s.batch, s.num_q_heads, s.head_dim)
            or tuple(bounds) != (s.num_blocks, s.num_kv_heads, BOUNDS_BYTES)
            or tuple(block_tables) != (s.batch, s.max_blocks_per_seq) or n_lens != s.batch):
        raise ValueError("q, bounds, block_tables or context_lens do not match the shape descriptor")
    if (tuple(selected) != (s.batch, s.num_kv_heads, s.max_pages)
            or tuple(selected_lens) != (s.batch, s.num_kv_heads)):
        raise ValueError("selected must be [B, Hkv, max_pages], selected_lens [B, Hkv]")
    return True


def xqa_select(q, bounds, block_tables, context_lens, max_pages: int = 0, first_pages: int = 1,
               last_pages: int = 1, selected=None, selected_lens=None, workspace=None,
               shape: XqaSelectShape | None = None, stream=None):
    """Choose the pages that each sequence's new token reads, for each kv head. q: fp16 [B, Hq,
    128]; bounds: uint8 [NB, Hkv, 272] (xqa_page_bounds); block_tables int32 [B, MBS];
    context_lens int32 [B]. Of a sequence with more than ``max_pages`` pages the first
    ``first_pages`` and last ``last_pages`` are taken, and of the others those with the
    highest scores (see include/xqa.h). Returns (selected int32 [B, Hkv, max_pages], -1
    behind the last page, and selected_lens int32 [B, Hkv]) for xqa_decode_selected."""
    if shape is None:
        shape = make_select_shape(q, bounds, block_tables, max_pages, first_pages, last_pages)
    fits = False
    try:  # the usual call, without a function call for each tensor
        dev = q.get_device()
        if (dev >= 0 and torch._C._cuda_getDevice() == dev and q.dtype is _F16 and q.is_contiguous()
                and bounds.dtype is _U8 and bounds.get_device() == dev and bounds.is_contiguous()
                and _all_i32(dev, block_tables, context_lens)):
            if selected is None:
                selected = _like(context_lens, (shape.batch, shape.num_kv_heads,
                                                max(shape.max_pages, 0)), stream)
            if selected_lens is None:
                selected_lens = _like(context_lens, (shape.batch, shape.num_kv_heads), stream)
            if workspace is None:
                with _allocating(stream):
                    workspace = alloc_select_workspace(shape, q.device)
            fits = _all_i32(dev, selected, selected_lens) and _select_fits(
                bytes(shape), q.shape, bounds.shape, block_tables.shape, context_lens.numel(),
                selected.shape, selected_lens.shape)
    except AttributeError:
        pass
    if not fits:
        _on_current((q, _F16, "q"), (bounds, _U8, "bounds"), (block_tables, _I32, "block_tables"),
                    (context_lens, _I32, "context_lens"),
                    *[(t, _I32, n) for t, n in ((selected, "selected"), (selected_lens, "selected_lens"))
                      if t is not None])
        raise ValueError("invalid arguments")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    code = load_library().xqa_select(
        q.data_ptr(), bounds.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
        selected.data_ptr(), selected_lens.data_ptr(), ctypes.byref(shape),
        _on(workspace, _U8, dev, "workspace"), workspace.numel(), handle)
    if code:
        raise XqaError(code, "xqa_select")
    return selected, selected_lens


def make_selected_shape(q, k_cache, selected, sm_scale: float = 0.0, max_ctas: int = 0,
                        min_pages_per_cta: int = 0, merge_mode: int = 0, kv_dtype: str = "e5m2",
                        kv_layout: str = "hnd") -> XqaShape:
    """Shape descriptor of xqa_decode_selected from q [B, Hq, 128], k_cache and selected [B,
    Hkv, K]; for alloc_workspace too."""
    if selected.dim() != 3 or q.dim() != 3:
        raise ValueError("q must be [B, Hq, 128], selected [B, Hkv, K]")
    shape = make_shape(q, k_cache, selected[:, 0], sm_scale, max_ctas, min_pages_per_cta, merge_mode,
                       kv_dtype, kv_layout)
    if selected.shape[1] != shape.num_kv_heads:
        raise ValueError("selected must have a row for each kv head")
    return shape


@functools.lru_cache(maxsize=1024)
def _selected_fits(shape: bytes, q, k_cache, v_cache, selected, selected_lens, n_out) -> bool:
    """Raises unless tensors of these shapes are what the descriptor says."""
    s = XqaShape.from_buffer_copy(shape)
    if (tuple(selected) != (s.batch, s.num_kv_heads, s.max_blocks_per_seq)
            or tuple(selected_lens) != (s.batch, s.num_kv_heads)):
        raise ValueError("selected or selected_lens does not match the shape descriptor")
    if len(q) != 3:
        raise ValueError("q must be [B, Hq, 128]: one new token for each sequence")
    return _decode_fits(shape, q, k_cache, v_cache, selected[::2], s.batch, n_out)


def xqa_decode_selected(q, k_cache, v_cache, selected, selected_lens, k_scale, v_scale, out=None,
                        workspace=None, shape: XqaShape | None = None, stream=None,
                        sm_scale: float = 0.0, max_ctas: int = 0, min_pages_per_cta: int = 0,
                        kv_dtype: str = "e5m2", kv_layout: str = "hnd"):
    """xqa_decode over a table of its own for each (sequence, kv head): selected int32 [B, Hkv,
    K] and selected_lens int32 [B, Hkv] (xqa_select) in place of block_tables and
    context_lens. q: fp16 [B, Hq, 128]. Returns ``out``, like q."""
    if shape is None:
        shape = make_selected_shape(q, k_cache, selected, sm_scale, max_ctas, min_pages_per_cta,
                                    kv_dtype=kv_dtype, kv_layout=kv_layout)
    fresh = out is None
    if fresh:
        out = _like(q, q.shape, stream)
    if workspace is None:
        with _allocating(stream):
            workspace = alloc_workspace(shape, q.device)
    fits = False
    try:  # the usual call, without a function call for each tensor
        dev = q.get_device()
        if (dev >= 0 and torch._C._cuda_getDevice() == dev and q.dtype is _F16 and q.is_contiguous()
                and k_cache.dtype is _U8 and k_cache.get_device() == dev and k_cache.is_contiguous()
                and v_cache.dtype is _U8 and v_cache.get_device() == dev and v_cache.is_contiguous()
                and (fresh or (out.dtype is _F16 and out.get_device() == dev and out.is_contiguous()))
                and workspace.dtype is _U8 and workspace.get_device() == dev and workspace.is_contiguous()
                and _all_i32(dev, selected, selected_lens)):
            fits = _selected_fits(bytes(shape), q.shape, k_cache.shape, v_cache.shape, selected.shape,
                                  selected_lens.shape, None if fresh else out.numel())
    except AttributeError:
        pass
    if not fits:
        _on_current((q, _F16, "q"), (k_cache, _U8, "k_cache"), (v_cache, _U8, "v_cache"),
                    (selected, _I32, "selected"), (selected_lens, _I32, "selected_lens"),
                    (out, _F16, "out"), (workspace, _U8, "workspace"))
        raise ValueError("invalid arguments")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _device_stream(stream)[1]
    ks, ksp = (k_scale, None) if type(k_scale) is float else _scale_arg(k_scale, dev, "k_scale")
    vs, vsp = (v_scale, None) if type(v_scale) is float else _scale_arg(v_scale, dev, "v_scale")
    if (ksp is None) != (vsp is None):
        raise ValueError("k_scale and v_scale must both be numbers, or both CUDA tensors")
    code = load_library().xqa_decode_selected(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), selected.data_ptr(), selected_lens.data_ptr(),
        ks, vs, ksp, vsp, out.data_ptr(), ctypes.byref(shape), workspace.data_ptr(), workspace.numel(), handle)
    if code:
        raise XqaError(code, "xqa_decode_selected")
    return out


def xqa_read_status(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(-1)
    _check(load_library().xqa_read_status(_cuda(workspace, torch.uint8, "workspace"),
                                          ctypes.byref(v), _stream_handle(stream)),
           "xqa_read_status")
    return int(v.value)


def xqa_read_plan(workspace: torch.Tensor, shape: XqaShape, stream=None) -> dict:
    import numpy as np

    nseg = shape.batch * shape.num_kv_heads
    header = np.zeros(4, np.int32)
    seg_start = np.zeros(nseg + 1, np.int32)
    seg_bad = np.zeros(nseg, np.int32)
    seg_cost = np.zeros(nseg, np.int32)
    _check(load_library().xqa_read_plan(_cuda(workspace, torch.uint8, "workspace"),
                                        ctypes.byref(shape), header.ctypes.data,
                                        seg_start.ctypes.data, seg_bad.ctypes.data,
                                        seg_cost.ctypes.data, _stream_handle(stream)),
           "xqa_read_plan")
    return {"ctas_launched": int(header[0]), "num_ctas": int(header[1]), "total_pages": int(header[2]),
            "num_segments": int(header[3]), "seg_start": seg_start, "seg_bad": seg_bad,
            "seg_cc": seg_cost}


def xqa_decode_static_workspace(q, k_cache, v_cache, block_tables, context_lens, k_scale: float,
                                v_scale: float, out=None, shape: XqaShape | None = None,
                                stream=None, sm_scale: float = 0.0, max_ctas: int = 0,
                                min_pages_per_cta: int = 0, merge_mode: int = 0,
                                kv_dtype: str = "e5m2", kv_layout: str = "hnd"):
    """xqa_decode without a workspace argument, for callers that may not allocate
    device memory: the scratch is the library's fixed per-device array (see
    include/xqa.h). q may be [B, Hq, D] or [B, T, Hq, D] (T new tokens per
    sequence). Calls that may overlap on one device must be ordered."""
    if shape is None:
        shape = make_shape(q, k_cache, block_tables, sm_scale, max_ctas, min_pages_per_cta,
                           merge_mode, kv_dtype=kv_dtype, kv_layout=kv_layout)
    if out is None:
        out = torch.empty_like(q)
    ptrs = _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, None, shape,
                        static=True)
    _check(load_library().xqa_decode_static_workspace(
        ptrs[0], ptrs[1], ptrs[2], ptrs[3], ptrs[4], float(k_scale), float(v_scale), ptrs[5],
        ctypes.byref(shape), _stream_handle(stream)), "xqa_decode_static_workspace")
    return out


def xqa_selftest_wait_timeout(budget_ns: int, stream=None) -> int:
    """Run the bounded-wait self-check (a wait nothing completes); returns the
    status the kernel wrote (XQA_ERR_DEVICE_TIMEOUT when the wait gave up)."""
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _check(load_library().xqa_selftest_wait_timeout(status.data_ptr(), int(budget_ns),
                                                    _stream_handle(stream)),
           "xqa_selftest_wait_timeout")
    torch.cuda.synchronize()
    return int(status.item())

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
``xqa_gather``, ``xqa_prefill``, ``xqa_prefill_workspace_size``.
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
)

KV_DTYPES = {"e5m2": 0, "e4m3": 1, "e2m1": 4}
KV_LAYOUTS = {"hnd": 0, "nhd": 1}
#: bytes of a (page, kv head) slice of a 4-bit cache (XQA_E2M1_SLICE_BYTES)
E2M1_SLICE_BYTES = 1152
ROW_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


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


class XqaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {xqa_status_string(code)} (status {code})")


_lib = None

_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_SHAPE = ctypes.POINTER(XqaShape)
_ROWS = ctypes.POINTER(XqaRows)
_PREFILL = ctypes.POINTER(XqaPrefillShape)
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
    return int(stream.cuda_stream)


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


def _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, workspace, shape):
    return (
        _cuda(q, torch.float16, "q"),
        _cuda(k_cache, torch.uint8, "k_cache"),
        _cuda(v_cache, torch.uint8, "v_cache"),
        _cuda(block_tables, torch.int32, "block_tables"),
        _cuda(context_lens, torch.int32, "context_lens"),
        _cuda(out, torch.float16, "out"),
        _cuda(workspace, torch.uint8, "workspace"),
    )


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
    if out is None or workspace is None:
        with _allocating(stream):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = alloc_workspace(shape, q.device)
    a = _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, workspace, shape)
    lib = load_library()
    if isinstance(k_scale, torch.Tensor) or isinstance(v_scale, torch.Tensor):
        ks = _cuda(k_scale, torch.float32, "k_scale")
        vs = _cuda(v_scale, torch.float32, "v_scale")
        _check(lib.xqa_decode_device_scales(a[0], a[1], a[2], a[3], a[4], ks, vs, a[5],
                                            ctypes.byref(shape), a[6], workspace.numel(),
                                            _stream_handle(stream)), "xqa_decode_device_scales")
        return out
    _check(lib.xqa_decode(a[0], a[1], a[2], a[3], a[4], float(k_scale), float(v_scale), a[5],
                          ctypes.byref(shape), a[6], workspace.numel(), _stream_handle(stream)),
           "xqa_decode")
    return out


def xqa_plan(context_lens, workspace, shape: XqaShape, stream=None) -> None:
    _check(load_library().xqa_plan(_cuda(context_lens, torch.int32, "context_lens"),
                                   ctypes.byref(shape), _cuda(workspace, torch.uint8, "workspace"),
                                   workspace.numel(), _stream_handle(stream)), "xqa_plan")


def xqa_attend_partial(q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, out,
                       workspace, shape: XqaShape, stream=None) -> None:
    a = _decode_args(q, k_cache, v_cache, block_tables, context_lens, out, workspace, shape)
    _check(load_library().xqa_attend_partial(a[0], a[1], a[2], a[3], a[4], float(k_scale),
                                             float(v_scale), a[5], ctypes.byref(shape), a[6],
                                             workspace.numel(), _stream_handle(stream)),
           "xqa_attend_partial")


def xqa_combine(context_lens, v_scale, out, workspace, shape: XqaShape, stream=None) -> None:
    _check(load_library().xqa_combine(_cuda(context_lens, torch.int32, "context_lens"),
                                      float(v_scale), _cuda(out, torch.float16, "out"),
                                      ctypes.byref(shape),
                                      _cuda(workspace, torch.uint8, "workspace"),
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


def _allocating(stream):
    """Context in which the binding allocates what a call on ``stream`` writes: the
    memory (and the zero fill of a workspace) belongs to that stream."""
    return torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream) else contextlib.nullcontext()


def _device_stream(stream):
    """(current device, handle of ``stream`` or of its current stream). The
    library works on the current device: the stream must be there, and every
    tensor (checked where its pointer is taken)."""
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
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
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    if n == 0 or h == 0:
        return h * d, d
    rs, hs, es = t.stride()
    if h == 1:
        hs = d
    if n == 1:
        rs = h * d
    if (es != 1 and d > 1) or rs <= 0 or hs <= 0:
        raise ValueError(f"{name}: the last dim must be contiguous and no stride may be 0")
    return rs, hs


def _cache_dims(cache: torch.Tensor, kv_dtype: str, kv_layout: str):
    """(num_blocks, num_kv_heads, block_size) of a cache tensor."""
    if kv_dtype == "e2m1":
        if cache.dim() != 3 or cache.shape[2] != E2M1_SLICE_BYTES or kv_layout != "hnd":
            raise ValueError("an e2m1 cache is [num_blocks, num_kv_heads, 1152], kv_layout 'hnd'")
        return cache.shape[0], cache.shape[1], 16
    if cache.dim() != 4:
        raise ValueError("an FP8 cache has four dims")
    nb, a, b, d = cache.shape
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


@functools.lru_cache(maxsize=256)
def _rows_descriptor(*fields) -> XqaRows:
    return XqaRows(*fields)


def _move_rows(fn_name, k, v, cu_seqlens, k_cache, v_cache, block_tables, context_lens, k_scale,
               v_scale, kv_dtype, kv_layout, status, stream):
    krs, khs = _heads(k, "k")  # CPU tensors are refused before CUDA is asked
    vrs, vhs = _heads(v, "v", k.dtype)
    dev, handle = _device_stream(stream)
    nb, hkv, bs = _cache_dims(k_cache, kv_dtype, kv_layout)
    n, h, d = k.shape
    b = context_lens.numel()
    if (v.shape != k.shape or v_cache.shape != k_cache.shape or h != hkv or d != 128
            or block_tables.dim() != 2 or block_tables.shape[0] != b
            or cu_seqlens.numel() != b + 1):
        raise ValueError("inconsistent rows / cache / block_tables / cu_seqlens shapes")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"k and v must be on the current device, cuda:{dev}")
    rows = _rows_descriptor(b, hkv, 128, bs, block_tables.shape[1], nb, n, KV_DTYPES[kv_dtype],
                            KV_LAYOUTS[kv_layout], ROW_DTYPES[k.dtype], krs, khs, vrs, vhs)
    kp, vp = k.data_ptr(), v.data_ptr()
    kc = _on(k_cache, torch.uint8, dev, "k_cache")
    vc = _on(v_cache, torch.uint8, dev, "v_cache")
    ks, ksp = _scale_arg(k_scale, dev, "k_scale")
    vs, vsp = _scale_arg(v_scale, dev, "v_scale")
    a = (kp, vp, kc, vc) if fn_name == "xqa_append" else (kc, vc, kp, vp)
    code = getattr(load_library(), fn_name)(
        a[0], a[1], _on(cu_seqlens, torch.int32, dev, "cu_seqlens"),
        _on(block_tables, torch.int32, dev, "block_tables"),
        _on(context_lens, torch.int32, dev, "context_lens"), ks, vs, ksp, vsp, a[2], a[3],
        ctypes.byref(rows), None if status is None else _on(status, torch.int32, dev, "status"),
        handle)
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
        with _allocating(stream):
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


def xqa_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k=None, out=None, lse=None, workspace=None,
                shape: XqaPrefillShape | None = None, stream=None, causal: bool = True,
                sm_scale: float = 0.0, max_ctas: int = 0):
    """Attention of whole prompts, packed by sequence: q fp16 or bf16 [total_q,
    Hq, 128], k and v [total_k, Hkv, 128], cu_seqlens_q / cu_seqlens_k int32
    [B+1] (keys default to the queries' offsets). With ``causal`` the last query
    of a sequence sees all its keys and each one before it one key less. ``lse``
    (fp32 [total_q, Hq], optional) receives the log-sum-exp. Returns ``out``;
    rows that see nothing are zero, rows behind the last sequence are not
    written."""
    if shape is None:
        shape = make_prefill_shape(q, k, v, cu_seqlens_q, causal, sm_scale, max_ctas, out)
    else:
        s = shape
        if _prefill_strides(q, k, v) != (s.q_row_stride, s.q_head_stride, s.k_row_stride,
                                         s.k_head_stride, s.v_row_stride, s.v_head_stride) or (
                s.total_q, s.num_q_heads, s.head_dim, s.total_k, s.num_kv_heads, s.dtype) != (
                *q.shape, k.shape[0], k.shape[1], ROW_DTYPES[q.dtype]):
            raise ValueError("q, k, v do not match the shape descriptor")
    dev, handle = _device_stream(stream)  # CPU tensors are refused before CUDA is asked
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens_q
    if out is None:
        with _allocating(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if shape.out_row_stride not in (0, q.shape[1] * q.shape[2]) or (
                shape.out_head_stride not in (0, q.shape[2])):
            raise ValueError("the shape descriptor names strides of out: pass out")
    elif out.shape != q.shape or _heads(out, "out", q.dtype) != (
            shape.out_row_stride or shape.num_q_heads * 128, shape.out_head_stride or 128):
        raise ValueError("out does not match q or the shape descriptor")
    if workspace is None:
        with _allocating(stream):
            workspace = alloc_prefill_workspace(shape, q.device)
    if cu_seqlens_q.numel() != shape.batch + 1 or cu_seqlens_k.numel() != shape.batch + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have batch + 1 entries")
    lp = None
    if lse is not None:
        lp = _on(lse, torch.float32, dev, "lse")
        if lse.shape != q.shape[:2]:
            raise ValueError("lse must be [total_q, num_q_heads]")
    for x in (q, k, v, out):
        if x.get_device() != dev:
            raise ValueError(f"q, k, v and out must be on the current device, cuda:{dev}")
    code = load_library().xqa_prefill(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _on(cu_seqlens_q, torch.int32, dev, "cu_seqlens_q"),
        _on(cu_seqlens_k, torch.int32, dev, "cu_seqlens_k"), out.data_ptr(), lp,
        ctypes.byref(shape), _on(workspace, torch.uint8, dev, "workspace"), workspace.numel(),
        handle)
    if code:
        raise XqaError(code, "xqa_prefill")
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
    ptrs = (
        _cuda(q, torch.float16, "q"),
        _cuda(k_cache, torch.uint8, "k_cache"),
        _cuda(v_cache, torch.uint8, "v_cache"),
        _cuda(block_tables, torch.int32, "block_tables"),
        _cuda(context_lens, torch.int32, "context_lens"),
        _cuda(out, torch.float16, "out"),
    )
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

"""Host checks of xqa_prefill (no GPU: every call is refused before the first CUDA
call; the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from paged_fp8_kv_gqa_gb300 import build

PTRS = dict(q=0x10000, k=0x20000, v=0x30000, cq=0x40000, ck=0x50000, out=0x60000, ws=0x100000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return xqa.load_library()


def shape(**kw):
    f = dict(batch=2, num_q_heads=32, num_kv_heads=4, head_dim=128, total_q=100, total_k=150,
             dtype=0, causal=1, sm_scale=0.0, max_ctas=152)
    f.update(kw)
    return xqa.XqaPrefillShape(**f)


def call(lib, s, nbytes=1 << 20, **kw):
    p = {**PTRS, **kw}
    return lib.xqa_prefill(p["q"], p["k"], p["v"], p["cq"], p["ck"], p["out"], None,
                           ctypes.byref(s) if s is not None else None, p["ws"], nbytes, None)


def test_workspace_size(lib):
    n = xqa.xqa_prefill_workspace_size(shape())
    # header, merge tickets and status words of a decode workspace
    assert 64 + 12 * 1024 <= n < 16384 and n % 256 == 0
    assert n == xqa.xqa_prefill_workspace_size(shape(batch=4000, total_q=100000, max_ctas=9999))
    decode = xqa.XqaShape(1, 8, 1, 128, 16, 1, 1, 0.0, 1, 0)
    assert xqa.xqa_workspace_size(decode) >= n  # a decode workspace may serve both
    assert lib.xqa_prefill_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == xqa.XQA_ERR_NULL
    assert lib.xqa_prefill_workspace_size(ctypes.byref(shape()), None) == xqa.XQA_ERR_NULL


def test_shape_refusals(lib):
    for bad in (dict(head_dim=64), dict(batch=0), dict(num_q_heads=30), dict(num_kv_heads=0),
                dict(num_q_heads=516, num_kv_heads=4),      # G = 129
                dict(total_q=-1), dict(total_k=-1), dict(dtype=2), dict(causal=2),
                dict(max_ctas=-1), dict(sm_scale=float("inf")),
                dict(total_q=2**23), dict(total_k=2**31 - 1), dict(batch=2**25),
                dict(q_row_stride=4), dict(k_head_stride=100), dict(v_row_stride=-128),
                dict(k_row_stride=2**39), dict(out_row_stride=128), dict(out_head_stride=64)):
        assert call(lib, shape(**bad)) == xqa.XQA_ERR_SHAPE, bad
    assert call(lib, None) == xqa.XQA_ERR_NULL


def test_pointer_refusals(lib):
    for p in PTRS:
        assert call(lib, shape(), **{p: 0}) == xqa.XQA_ERR_NULL, p
    for p in ("q", "k", "v", "out"):
        assert call(lib, shape(), **{p: PTRS[p] + 8}) == xqa.XQA_ERR_ALIGN, p
    assert call(lib, shape(), ws=PTRS["ws"] + 128) == xqa.XQA_ERR_ALIGN
    assert call(lib, shape(), nbytes=xqa.xqa_prefill_workspace_size(shape()) - 1) == xqa.XQA_ERR_WORKSPACE
    assert call(lib, shape(total_q=0), q=0, out=0) == xqa.XQA_OK  # nothing to do
    assert xqa.xqa_status_string(xqa.XQA_ERR_BAD_OFFSETS) != "unknown status"


def test_binding_refuses_cpu_tensors_before_the_library():
    x = torch.zeros(3, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        xqa.xqa_prefill(x, x, x, torch.zeros(2, dtype=torch.int32))

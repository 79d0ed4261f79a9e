"""Host checks of xqa_extend (no GPU: every call is refused before the first CUDA call, or
returns before it; the addresses are never dereferenced)."""
import ctypes
import math

import pytest

import paged_fp8_kv_gqa_gb300 as xqa
from test_abi import lib  # noqa: F401

GOOD = dict(batch=4, num_q_heads=32, num_kv_heads=4, head_dim=128, block_size=16,
            max_blocks_per_seq=100, num_blocks=500, total_q=64, dtype=0, kv_dtype=0, kv_layout=0,
            causal=1, sm_scale=0.0, max_ctas=8)


def shape(**kw):
    return xqa.XqaExtendShape(**{**GOOD, **kw})


def call(lib, s, ptr=None, scales=(1.0, 1.0), nbytes=1 << 40):  # noqa: F811
    a = {n: 0x100000 * (i + 1) for i, n in enumerate(("q", "k", "v", "bt", "lens", "cu", "out", "ws"))}
    a.update(ptr or {})
    return lib.xqa_extend(a["q"], a["k"], a["v"], a["bt"], a["lens"], a["cu"], *scales, None, None,
                          a["out"], None, ctypes.byref(s) if s is not None else None, a["ws"], nbytes,
                          None)


BAD = [dict(batch=0), dict(batch=-1), dict(num_kv_heads=0), dict(num_q_heads=0), dict(num_q_heads=30),
       dict(num_q_heads=4 * 129), dict(head_dim=64), dict(block_size=32), dict(max_blocks_per_seq=0),
       dict(max_blocks_per_seq=2**27), dict(num_blocks=0), dict(num_blocks=2**28), dict(total_q=-1),
       dict(total_q=2**23), dict(dtype=2), dict(kv_dtype=2), dict(kv_layout=2),
       dict(kv_dtype=4, kv_layout=1), dict(causal=2), dict(max_ctas=-1), dict(sm_scale=math.inf),
       dict(q_row_stride=4), dict(q_row_stride=-8), dict(q_head_stride=12), dict(q_row_stride=2**61),
       dict(out_head_stride=64), dict(out_row_stride=128), dict(out_row_stride=2**60)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_shapes_that_are_refused(lib, bad):  # noqa: F811
    n = ctypes.c_size_t()
    assert call(lib, shape(**bad)) == xqa.XQA_ERR_SHAPE
    assert lib.xqa_extend_workspace_size(ctypes.byref(shape(**bad)), ctypes.byref(n)) == xqa.XQA_ERR_SHAPE


def test_pointers_sizes_and_scales(lib):  # noqa: F811
    s = shape()
    for name in ("q", "k", "v", "bt", "lens", "cu", "out", "ws"):
        assert call(lib, s, {name: None}) == xqa.XQA_ERR_NULL
    for name in ("q", "k", "v", "out"):
        assert call(lib, s, {name: 0x100008}) == xqa.XQA_ERR_ALIGN
    assert call(lib, s, {"ws": 0x100080}) == xqa.XQA_ERR_ALIGN
    assert call(lib, s, nbytes=xqa.xqa_extend_workspace_size(s) - 1) == xqa.XQA_ERR_WORKSPACE
    for bad in (0.0, -1.0, math.inf, math.nan):
        assert call(lib, s, scales=(bad, 1.0)) == xqa.XQA_ERR_VALUE
        assert call(lib, s, scales=(1.0, bad)) == xqa.XQA_ERR_VALUE
    assert call(lib, None) == xqa.XQA_ERR_NULL
    assert lib.xqa_extend_workspace_size(ctypes.byref(s), None) == xqa.XQA_ERR_NULL
    assert call(lib, shape(total_q=0), {"q": None, "out": None}) == xqa.XQA_OK


def test_workspace_grows_with_the_work(lib):  # noqa: F811
    small = xqa.xqa_extend_workspace_size(shape(batch=1, total_q=1, max_blocks_per_seq=1, max_ctas=152))
    large = xqa.xqa_extend_workspace_size(shape(max_ctas=152))
    assert small < large
    assert xqa.xqa_extend_workspace_size(shape(max_ctas=5000)) <= xqa.xqa_extend_workspace_size(
        shape(max_ctas=1024))

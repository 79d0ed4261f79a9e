"""Host checks of xqa_append and xqa_gather (no GPU: every call is refused before
the first CUDA call; the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from paged_fp8_kv_gqa_gb300 import build

K, V, CU, BT, LENS, KC, VC = (0x10000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return xqa.load_library()


def rows(**kw):
    f = dict(batch=2, num_kv_heads=4, head_dim=128, block_size=16, max_blocks_per_seq=8,
             num_blocks=64, num_rows=10, kv_dtype=0, kv_layout=0, dtype=0)
    f.update(kw)
    return xqa.XqaRows(**f)


def call(lib, name, r, k=K, v=V, cu=CU, bt=BT, lens=LENS, kc=KC, vc=VC, ks=1.0, vs=1.0):
    a, b = ((k, v), (kc, vc)) if name == "xqa_append" else ((kc, vc), (k, v))
    return getattr(lib, name)(*a, cu, bt, lens, ks, vs, None, None, *b,
                              ctypes.byref(r) if r is not None else None, None, None)


@pytest.mark.parametrize("name", ["xqa_append", "xqa_gather"])
def test_refusals(lib, name):
    assert call(lib, name, None) == xqa.XQA_ERR_NULL
    for bad in (dict(head_dim=64), dict(block_size=32), dict(batch=0), dict(num_kv_heads=0),
                dict(max_blocks_per_seq=0), dict(num_blocks=0), dict(num_rows=-1),
                dict(kv_dtype=2), dict(kv_dtype=3), dict(kv_layout=2), dict(dtype=2),
                dict(kv_dtype=4, kv_layout=1),              # 4 bits: HND only
                dict(num_blocks=2**25 + 1),                 # pool rows past int32
                dict(num_rows=2**29),                       # rows x heads past int32
                dict(k_row_stride=4), dict(v_head_stride=12), dict(k_head_stride=-128)):
        assert call(lib, name, rows(**bad)) == xqa.XQA_ERR_SHAPE, bad
    for ptr in ("k", "v", "cu", "bt", "lens", "kc", "vc"):
        assert call(lib, name, rows(), **{ptr: 0}) == xqa.XQA_ERR_NULL, ptr
    for ptr in ("k", "v", "kc", "vc"):
        assert call(lib, name, rows(), **{ptr: 0x10008}) == xqa.XQA_ERR_ALIGN, ptr
    assert call(lib, name, rows(num_rows=0), k=0, v=0) == xqa.XQA_OK  # nothing to do


def test_scales_of_append(lib):
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert call(lib, "xqa_append", rows(), ks=bad) == xqa.XQA_ERR_VALUE
        assert call(lib, "xqa_append", rows(), vs=bad) == xqa.XQA_ERR_VALUE
    assert xqa.xqa_status_string(xqa.XQA_ERR_VALUE) != "unknown status"


def test_written_rows_must_not_overlap(lib):
    for bad in (dict(k_row_stride=128), dict(v_row_stride=256, v_head_stride=128),
                dict(k_head_stride=64)):
        assert call(lib, "xqa_gather", rows(**bad)) == xqa.XQA_ERR_SHAPE, bad


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(3, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        xqa.xqa_append(cpu, cpu, None, None, None, None, None, 1.0, 1.0)
    with pytest.raises(ValueError, match="e2m1"):
        xqa._cache_dims(torch.zeros(2, 2, 16, 72, dtype=torch.uint8), "e2m1", "hnd")
    with pytest.raises(ValueError, match="e2m1"):
        xqa._cache_dims(torch.zeros(2, 2, 1152, dtype=torch.uint8), "e2m1", "nhd")

"""Host checks of the calls over pages, bounds and choices (no GPU: every call is refused
before the first CUDA call, or returns before it; the addresses are never dereferenced)."""
import ctypes

import pytest

import paged_fp8_kv_gqa_gb300 as xqa
from test_abi import lib  # noqa: F401

PTR = [0x100000 * (i + 1) for i in range(10)]


def pages(**kw):
    return xqa.XqaPages(**{**dict(batch=4, block_size=16, max_blocks_per_seq=100, num_blocks=500, num_rows=64), **kw})


def assign(lib, s, ptr=PTR):  # noqa: F811
    return lib.xqa_assign_pages(*ptr, ctypes.byref(s) if s is not None else None, None, None)


def release(lib, s, ptr=PTR[:7]):  # noqa: F811
    return lib.xqa_release_pages(*ptr, ctypes.byref(s) if s is not None else None, None, None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(batch=16385), dict(block_size=32), dict(max_blocks_per_seq=0),
                                 dict(max_blocks_per_seq=2**27), dict(num_blocks=0), dict(num_blocks=2**27),
                                 dict(num_rows=-1), dict(num_rows=2**30), dict(batch=16384, max_blocks_per_seq=2**17)],
                         ids=str)
def test_pages_that_are_refused(lib, bad):  # noqa: F811
    assert assign(lib, pages(**bad)) == xqa.XQA_ERR_SHAPE
    assert release(lib, pages(**bad)) == xqa.XQA_ERR_SHAPE


def test_pointers_of_page_calls(lib):  # noqa: F811
    assert assign(lib, None) == release(lib, None) == xqa.XQA_ERR_NULL
    for i in range(8):
        assert assign(lib, pages(), [None if j == i else p for j, p in enumerate(PTR)]) == xqa.XQA_ERR_NULL
    for i in range(7):
        assert release(lib, pages(), [None if j == i else p for j, p in enumerate(PTR[:7])]) == xqa.XQA_ERR_NULL


ROWS = dict(batch=4, num_kv_heads=4, head_dim=128, block_size=16, max_blocks_per_seq=100, num_blocks=500,
            num_rows=64, kv_dtype=0, kv_layout=0)


def bounds(lib, s, ptr=PTR[:5]):  # noqa: F811
    return lib.xqa_page_bounds(*ptr, ctypes.byref(s) if s is not None else None, None, None)


def test_bounds_calls_that_are_refused(lib):  # noqa: F811
    for bad in (dict(batch=0), dict(num_kv_heads=0), dict(head_dim=64), dict(block_size=8), dict(max_blocks_per_seq=0),
                dict(num_blocks=0), dict(num_blocks=2**25), dict(num_rows=-1), dict(num_rows=2**29), dict(kv_dtype=3),
                dict(kv_layout=2), dict(kv_dtype=4, kv_layout=1)):
        assert bounds(lib, xqa.XqaRows(**{**ROWS, **bad})) == xqa.XQA_ERR_SHAPE, bad
    good = xqa.XqaRows(**ROWS)
    for i in range(5):
        assert bounds(lib, good, [None if j == i else p for j, p in enumerate(PTR[:5])]) == xqa.XQA_ERR_NULL
    assert bounds(lib, good, [PTR[0] + 8, *PTR[1:5]]) == xqa.XQA_ERR_ALIGN
    assert bounds(lib, good, [*PTR[:4], PTR[4] + 8]) == xqa.XQA_ERR_ALIGN
    assert bounds(lib, None) == xqa.XQA_ERR_NULL
    assert bounds(lib, xqa.XqaRows(**{**ROWS, "num_rows": 0}), [None] * 5) == xqa.XQA_OK


SELECT = dict(batch=4, num_q_heads=32, num_kv_heads=4, head_dim=128, block_size=16, max_blocks_per_seq=100,
              num_blocks=500, max_pages=20, first_pages=1, last_pages=2, max_ctas=8)


def select(lib, s, ptr=PTR[:6], ws=PTR[6], nbytes=1 << 40):  # noqa: F811
    return lib.xqa_select(*ptr, ctypes.byref(s) if s is not None else None, ws, nbytes, None)


def test_choices_that_are_refused(lib):  # noqa: F811
    n = ctypes.c_size_t()
    for bad in (dict(batch=0), dict(num_kv_heads=0), dict(num_q_heads=0), dict(num_q_heads=30), dict(num_q_heads=68),
                dict(head_dim=64), dict(block_size=32), dict(max_blocks_per_seq=0), dict(num_blocks=0),
                dict(max_pages=0), dict(first_pages=-1), dict(last_pages=0), dict(first_pages=19),
                dict(first_pages=2**31 - 1), dict(max_ctas=-1), dict(batch=1, max_blocks_per_seq=2**24 + 1), dict(batch=2**20, max_blocks_per_seq=2**10),
                dict(batch=2**20, max_pages=2**10)):
        s = xqa.XqaSelectShape(**{**SELECT, **bad})
        assert select(lib, s) == xqa.XQA_ERR_SHAPE, bad
        assert lib.xqa_select_workspace_size(ctypes.byref(s), ctypes.byref(n)) == xqa.XQA_ERR_SHAPE
    good = xqa.XqaSelectShape(**SELECT)
    for i in range(6):
        assert select(lib, good, [None if j == i else p for j, p in enumerate(PTR[:6])]) == xqa.XQA_ERR_NULL
    assert select(lib, good, ws=None) == xqa.XQA_ERR_NULL
    assert select(lib, good, ws=PTR[6] + 128) == xqa.XQA_ERR_ALIGN
    assert select(lib, good, [PTR[0] + 2, *PTR[1:6]]) == xqa.XQA_ERR_ALIGN
    assert select(lib, good, [PTR[0], PTR[1] + 8, *PTR[2:6]]) == xqa.XQA_ERR_ALIGN
    assert select(lib, good, nbytes=xqa.xqa_select_workspace_size(good) - 1) == xqa.XQA_ERR_WORKSPACE


def test_decode_of_selected_pages_refuses(lib):  # noqa: F811
    shape = xqa.XqaShape(16, 32, 4, 128, 16, 20, 500, 0.0, 152, 0)
    size = xqa.xqa_workspace_size(shape)

    def call(ptr=PTR[:5], scales=(None, None), out=PTR[5], s=shape, nbytes=size):
        return lib.xqa_decode_selected(*ptr, 1.0, 1.0, *scales, out, ctypes.byref(s), PTR[6], nbytes, None)

    for i in range(5):
        assert call([None if j == i else p for j, p in enumerate(PTR[:5])]) == xqa.XQA_ERR_NULL
    assert call(out=None) == xqa.XQA_ERR_NULL
    assert call(scales=(PTR[7], None)) == call(scales=(None, PTR[7])) == xqa.XQA_ERR_NULL
    assert call(nbytes=size - 1) == xqa.XQA_ERR_WORKSPACE
    assert call([PTR[0] + 2, *PTR[1:5]]) == xqa.XQA_ERR_ALIGN
    several = xqa.XqaShape(16, 32, 4, 128, 16, 20, 500, 0.0, 152, 0, 0, 0, 0, 2)
    assert call(s=several, nbytes=1 << 40) == xqa.XQA_ERR_SHAPE


def test_status_string_of_the_pool(lib):  # noqa: F811
    assert "pages" in xqa.xqa_status_string(xqa.XQA_ERR_NO_PAGES)

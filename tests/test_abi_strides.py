"""Host checks of strides whose offsets pass 64 bits (no GPU: every call is refused before the
first CUDA call; the addresses are never dereferenced)."""
import ctypes

import pytest

import paged_fp8_kv_gqa_gb300 as xqa
from test_abi_prefill import call as prefill_call, lib, shape  # noqa: F401
from test_abi_rows import call, rows


@pytest.mark.parametrize("name", ["xqa_append", "xqa_gather"])
@pytest.mark.parametrize("side", ["k", "v"])
def test_rows(lib, name, side):  # noqa: F811
    for n, rs, hs in ((2**28, 2**39, 2**38),   # the last row's offset wraps around to a small one
                      (2**28, 2**33, 128), (2, 2**60, 128), (1, 8, 2**59), (3, 2**62, 0)):
        r = rows(num_rows=n, **{side + "_row_stride": rs, side + "_head_stride": hs})
        assert call(lib, name, r) == xqa.XQA_ERR_SHAPE, (n, rs, hs)


def test_prompt_attention(lib):  # noqa: F811
    for side in ("k", "v"):
        s = shape(total_k=2**30, **{side + "_row_stride": 2**37})
        assert prefill_call(lib, s, nbytes=1 << 40) == xqa.XQA_ERR_SHAPE
        n = ctypes.c_size_t()
        assert lib.xqa_prefill_workspace_size(ctypes.byref(s), ctypes.byref(n)) == xqa.XQA_ERR_SHAPE
    big = shape(total_k=2**22, k_row_stride=2**37)
    assert xqa.xqa_prefill_workspace_size(big) > 0  # still within 64 bits

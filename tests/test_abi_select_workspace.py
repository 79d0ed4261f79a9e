"""Where xqa_select keeps its tickets and keys (no GPU: sizes only). Tickets outlive a call, so
they have to lie where no shape's keys do: within the part that is the same for all shapes."""
import ctypes

import pytest

import paged_fp8_kv_gqa_gb300 as xqa
from test_abi import lib  # noqa: F401

FIXED = 12544  # header, tickets and status words of every call's workspace, in whole 256 bytes


@pytest.mark.parametrize("batch,hkv,mbs", [(1, 1, 1), (1, 8, 8192), (3, 2, 1001), (64, 4, 1100), (500, 4, 37)])
def test_keys_begin_at_one_place(lib, batch, hkv, mbs):  # noqa: F811
    s = xqa.XqaSelectShape(batch, 8 * hkv, hkv, 128, 16, mbs, 500, 20, 1, 2, 152)
    n = ctypes.c_size_t()
    assert lib.xqa_select_workspace_size(ctypes.byref(s), ctypes.byref(n)) == xqa.XQA_OK
    assert n.value == FIXED + 4 * batch * hkv * ((mbs + 3) // 4 * 4)


@pytest.mark.parametrize("max_ctas", [1, 7, 304, 1024, 5000])
def test_tickets_fit_their_place(max_ctas):
    """Segments of several chunks: at most half of the CTAs, whatever the batch."""
    ctas = min(max_ctas, 1024)
    several = [nseg for nseg in range(1, 5000) if ctas // nseg > 1]
    assert len(several) <= 1024 // 2 and max(several, default=0) <= 2 * 1024

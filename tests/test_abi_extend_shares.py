"""The most CTAs that xqa_extend launches (no GPU: its workspace has room for their pieces) against
the shares that the kernel's own line of work has for given lengths. Sequences hold their new
tokens, as a cache does (one that does not has hidden keys on the line, which need no CTA)."""
import ctypes
import random

import pytest

import paged_fp8_kv_gqa_gb300 as xqa
from test_abi import lib  # noqa: F401

SHARE, UNIT, KEY = 384, 256, 16  # keys; a key of a unit of two row tiles is 16 long, of one 10 or 12


def ctas_of(lib, batch, hq, hkv, mbs, total_q, max_ctas):  # noqa: F811
    s = xqa.XqaExtendShape(batch, hq, hkv, 128, 16, mbs, 100000, total_q, 0, 0, 0, 1, 0.0, max_ctas)
    n = ctypes.c_size_t()
    assert lib.xqa_extend_workspace_size(ctypes.byref(s), ctypes.byref(n)) == xqa.XQA_OK
    # a fixed part, a few words for each CTA, and its two pieces of 256 rows of 128 + 2 floats
    return (n.value - 12544) // (2 * 256 * 130 * 4)


def line_shares(new, ctx, hq, hkv, causal, key_one):
    t = 128 // (hq // hkv)
    line = 0
    for n, c in zip(new, ctx):
        units = -(-n // (2 * t))
        for i in range(units):
            sees = max(0, c - n) + min(2 * t * (i + 1), n) if causal else c
            one = i == units - 1 and n - 2 * t * i <= t
            line += UNIT * KEY + (key_one if one else KEY) * sees
    return max(1, line * hkv // (SHARE * KEY))


@pytest.mark.parametrize("batch,hq,hkv,mbs,new,want", [(64, 8, 1, 1, 1, 44), (4, 8, 1, 8, 5, 4)])
def test_short_tables(lib, batch, hq, hkv, mbs, new, want):  # noqa: F811
    """Single tokens over one page, a few over eight: as many CTAs as the line has shares for."""
    full = line_shares([new] * batch, [16 * mbs] * batch, hq, hkv, True, 10)
    assert full >= want - 1
    assert ctas_of(lib, batch, hq, hkv, mbs, batch * new, 152) >= full


def test_no_line_has_more_shares(lib):  # noqa: F811
    r = random.Random(4)
    for _ in range(300):
        hkv = r.choice([1, 2, 4, 8])
        hq = hkv * r.choice([1, 3, 8, 16, 33, 128])
        mbs, batch = r.choice([1, 2, 8, 9, 60]), r.choice([1, 2, 5, 33])
        new = [r.choice([0, 1, 2, 17, 300]) for _ in range(batch)]
        if not sum(new):
            continue
        new = [min(n, 16 * mbs) for n in new]
        ctx = [r.randint(n, 16 * mbs) for n in new]
        got = ctas_of(lib, batch, hq, hkv, mbs, sum(new), 152)
        for causal in (True, False):
            for key_one in (10, 12):
                assert got >= min(152, line_shares(new, ctx, hq, hkv, causal, key_one))

"""xqa_prefill where one CTA works through units with and without keys, and where a row has
infinities or NaN in one piece of its keys (see test_gpu_prefill for the bounds)."""
import math

import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_prefill import Call, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("max_ctas", [1, 2, 0])
@pytest.mark.parametrize("lq,lk", [([40, 7, 9, 20, 50], [40, 0, 0, 0, 50]),
                                   ([300, 200, 100, 1], [300, 0, 0, 0]),
                                   ([1, 2, 3, 4, 5, 6, 7, 8], [0, 0, 9, 0, 0, 0, 0, 700]),
                                   ([900], [30]), ([700, 5, 640], [129, 0, 260])])
def test_units_without_keys_between_units_with_keys(lq, lk, max_ctas, causal):
    # sequences without keys, and causal rows in front of the first key: every CTA meets runs
    # of such units after, before and between those with work
    for hq, hkv in ((8, 2), (6, 1)):
        c = Call(lq, lk, hq=hq, hkv=hkv, seed=sum(lk), dtype="bf16" if hkv == 1 else "fp16")
        out = c.run(causal, max_ctas=max_ctas)
        c.check(out, causal)
        assert torch.equal(c.run(causal, max_ctas=max_ctas), out)


def test_many_more_queries_than_keys():
    c = Call([8192], [128], hq=32, hkv=4, seed=3, dtype="bf16")
    c.check(c.run())


@pytest.mark.parametrize("max_ctas", [1, 3])
def test_bad_key_offsets_between_good_sequences(max_ctas):
    lens = [70, 40, 30, 300, 20]
    c = Call(lens, hq=8, hkv=2, seed=4)
    want = c.run(max_ctas=max_ctas)
    good = c.ck.clone()
    c.ck[2:4] = torch.tensor([-1, -1], dtype=torch.int32)  # sequences 1, 2 and 3
    lse = torch.zeros_like(c.lse)
    out = torch.full_like(want, 9.0)
    xqa.xqa_prefill(c.q, c.k, c.v, c.cq, c.ck, out=out, lse=lse, workspace=c.ws, shape=c.shape)
    assert xqa.xqa_read_status(c.ws) == xqa.XQA_ERR_BAD_OFFSETS
    lost = slice(70, 440)
    assert bool(torch.isnan(out[lost]).all()) and bool(torch.isnan(lse[lost]).all())
    for keep in (slice(0, 70), slice(440, 460)):
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], c.lse[keep])
    xqa.xqa_prefill(c.q, c.k, c.v, c.cq, good, out=out, workspace=c.ws, shape=c.shape)
    assert torch.equal(out, want) and xqa.xqa_read_status(c.ws) == xqa.XQA_OK


@pytest.mark.parametrize("max_ctas", [1, 0])
def test_offsets_that_overlap_end_with_an_error(max_ctas):
    # 0, 200, 0, 200, ..., 240: every other sequence is the first one again; as many units as
    # ascending offsets can have are worked off, which leaves out the last sequence
    c = Call([200, 40], hq=8, hkv=2, seed=5)
    want = c.run(max_ctas=max_ctas)
    cu = (torch.arange(601, device="cuda") % 2 * 200).to(torch.int32)
    cu[600] = 240
    shape = xqa.make_prefill_shape(c.q, c.k, c.v, cu, max_ctas=max_ctas)
    ws = xqa.alloc_prefill_workspace(shape)
    for _ in range(2):
        out = torch.full_like(want, 7.0)
        xqa.xqa_prefill(c.q, c.k, c.v, cu, cu, out=out, workspace=ws, shape=shape)
        assert xqa.xqa_read_status(ws) == xqa.XQA_ERR_BAD_OFFSETS
        assert torch.equal(out[:200], want[:200]) and bool((out[200:] == 7.0).all())
        assert not bool(ws[16:64].any())  # counters back at zero
    xqa.xqa_prefill(c.q, c.k, c.v, c.cq, c.ck, out=out, workspace=ws)
    assert torch.equal(out, want) and xqa.xqa_read_status(ws) == xqa.XQA_OK


def same_specials(a, b):
    """NaN in the same places, equal infinities."""
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    inf = torch.isinf(b)
    assert torch.equal(torch.isinf(a), inf) and torch.equal(a[inf].double(), b[inf].double())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("at", [[256], [0, 256], range(128), range(128, 256), [100]])
def test_a_piece_of_nan_keys_makes_its_rows_nan(at, causal, dtype):
    # the second sequence's three tiles are a piece each, the last one of a single key; its
    # rows that see a NaN key are NaN, whole or in pieces
    for hq, hkv in ((8, 2), (5, 1)):
        c = Call([3, 2], [4000, 257], hq=hq, hkv=hkv, seed=7, dtype=dtype)
        for i in at:
            c.k[4000 + i] = math.nan
        out = c.run(causal)
        assert c.ws.numel() > 16384  # in pieces
        lse = c.lse.clone()
        sees = causal and list(at) == [256]  # then the first of the two rows sees none of them
        assert bool(torch.isnan(out[3 + sees:]).all()) and bool(torch.isnan(lse[3 + sees:]).all())
        assert bool(torch.isfinite(out[:3 + sees]).all()) and bool(torch.isfinite(lse[:3 + sees]).all())
        one = c.run(causal, max_ctas=1)
        assert c.ws.numel() < 16384  # whole
        same_specials(out, one)
        same_specials(lse, c.lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("val", [math.inf, -math.inf, math.nan])
def test_infinities_in_a_piece_of_little_weight(val, causal):
    # the last key's logits lie about 300 below the others: its weight is a number in 64 bits,
    # not in 32, and its value reaches every row that sees it
    c = Call([3, 2], [4000, 257], hq=8, hkv=2, seed=8)
    c.q[3:] = 1.0
    c.k[4000 + 256] = -300 * math.sqrt(128) / 128
    c.v[4000 + 256, :, 9] = val
    out = c.run(causal)
    assert c.ws.numel() > 16384
    c.check(out, causal)
    want, _, _ = plain(c.q, c.k, c.v, c.lq, c.lk, causal)
    assert int((~torch.isfinite(want)).sum()) == 8 * (1 if causal else 2)
    same_specials(out, want)


def test_a_unit_that_takes_longer_than_a_wait():
    # 2^27 keys (34 GB) for one CTA, 1.4 s of work: every role waits for as long as the others
    # get on. Equal weights, 2^20 values of 1: the sums are
    # exact, out is rounded twice (32 bits, then fp16)
    n = 2**27
    k = torch.zeros(n, 1, 128, dtype=torch.float16, device="cuda")
    k[2**26:2**26 + 2**20] = 1.0
    q = torch.zeros(3, 2, 128, dtype=torch.float16, device="cuda")
    cq, ck = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (3, n))
    shape = xqa.make_prefill_shape(q, k, k, cq, causal=False, max_ctas=1)
    ws = xqa.alloc_prefill_workspace(shape)
    out, lse = torch.zeros_like(q), torch.zeros(3, 2, device="cuda")
    xqa.xqa_prefill(q, k, k, cq, ck, out=out, lse=lse, workspace=ws, shape=shape)
    status = xqa.xqa_read_status(ws)
    del k
    torch.cuda.empty_cache()
    assert status == xqa.XQA_OK
    assert float((out.double() * n / 2**20 - 1).abs().max()) <= 2.0**-11 + 2.0**-22
    assert float((lse.double() - math.log(n)).abs().max()) <= 2.0**-18 * (1 + math.log(n))

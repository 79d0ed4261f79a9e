"""Pools of more than 2^32 bytes: the operators over the cache read and write the pages at their ends as
they do others. A few pages at the end and the beginning of large pools hold what a small pool holds;
results have to equal those over the small one bit for bit."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_extend import Cache, Call, i32
from test_gpu_prefill import offsets

pytestmark = pytest.mark.gpu


def moved(cache, large):
    """(k, v, table, place of each page of the small pool) of a pool of `large` pages whose last,
    middle and first pages are the small pool's."""
    n = cache.nb
    place = torch.empty(n, dtype=torch.long)
    place[0::3] = large - 1 - torch.arange(len(place[0::3]))
    place[1::3] = large // 2 + torch.arange(len(place[1::3]))
    place[2::3] = torch.arange(len(place[2::3]))
    place = place.cuda()
    pools = []
    for small in (cache.k, cache.v):
        pool = torch.full((large, *small.shape[1:]), 0x7F, dtype=torch.uint8, device="cuda")
        pool[place] = small
        assert pool.numel() > 2**32
        pools.append(pool)
    table = torch.where(cache.bt >= 0, place[cache.bt.clamp(min=0).long()].to(torch.int32), cache.bt)
    return *pools, table, place


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
def test_chunks_and_selected_pages(kv_dtype, kv_layout):
    c = Call([5, 1, 300], [900, 2500, 300], hq=8, hkv=2, kv_dtype=kv_dtype, kv_layout=kv_layout, seed=3)
    large = 2**21 if kv_dtype == "e2m1" else 2**20 + 77
    want, cache = c.run(), c.cache
    k, v, table, place = moved(cache, large)
    got = xqa.xqa_extend(c.q, k, v, table, cache.lens, c.cu, 1.0, 1.0, **cache.kind)
    assert torch.equal(got, want)
    # bounds, choice and attention over it
    small = xqa.alloc_bounds(cache.k, **cache.kind)
    bounds = torch.zeros((large, 2, 272), dtype=torch.uint8, device="cuda")
    for x, t, b in ((cache.k, cache.bt, small), (k, table, bounds)):
        xqa.xqa_page_bounds(x, t, cache.lens, offsets(cache.ctx), sum(cache.ctx), b, **cache.kind)
    assert torch.equal(bounds[place], small)
    q = c.q[:3].contiguous()
    picks = [xqa.xqa_select(q, b, t, cache.lens, 9, 1, 2) for b, t in ((small, cache.bt), (bounds, table))]
    at = torch.where(picks[0][0] >= 0, place[picks[0][0].clamp(min=0).long()].to(torch.int32), picks[0][0])
    assert torch.equal(picks[1][0], at) and torch.equal(picks[1][1], picks[0][1])
    outs = [xqa.xqa_decode_selected(q, a, b, *p, 1.0, 1.0, **cache.kind)
            for a, b, p in ((cache.k, cache.v, picks[0]), (k, v, picks[1]))]
    assert torch.equal(*outs)


def test_bounds_past_32_bit_offsets():
    """The bounds' own buffer past 2^32 bytes, of a 4-bit pool."""
    large = 2**24 + 5
    c = Cache([100, 40], 1, "e2m1", "hnd", seed=2)
    small = xqa.alloc_bounds(c.k, **c.kind)
    xqa.xqa_page_bounds(c.k, c.bt, c.lens, offsets(c.ctx), 140, small, **c.kind)
    k, _, table, place = moved(c, large)
    bounds = torch.zeros((large, 1, 272), dtype=torch.uint8, device="cuda")
    assert bounds.numel() > 2**32
    xqa.xqa_page_bounds(k, table, c.lens, offsets(c.ctx), 140, bounds, **c.kind)
    assert torch.equal(bounds[place], small)
    q = torch.randn(2, 4, 128, device="cuda").half()
    (a, la), (b, lb) = (xqa.xqa_select(q, x, t, c.lens, 3) for x, t in ((small, c.bt), (bounds, table)))
    assert torch.equal(b, torch.where(a >= 0, place[a.clamp(min=0).long()].to(torch.int32), a)) and torch.equal(la, lb)

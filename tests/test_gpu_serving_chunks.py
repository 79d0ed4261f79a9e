"""The operators together, as a server with one pool of pages uses them: requests get pages as
they grow and give them back when they end, prompts go through in chunks that attend over the
cache, and tokens are decoded over the pages that the bounds select.

Attention is held against float64 over the values that the cache holds (as its pages say,
through the tables that the operators made), with the tolerances of the operators' own tests.
"""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from gpu_helpers import ATOL, RTOL
from oracle import attention, e2m1
from test_gpu_extend import i32
from test_gpu_prefill import compare, offsets, plain
from test_gpu_select import plain_select

pytestmark = pytest.mark.gpu

HQ, HKV, PLACES, MBS, NB, ROWS = 8, 2, 4, 40, 90, 700
KS, VS = 0.5, 0.25


class Server:
    def __init__(self, kv_dtype, kv_layout, seed):
        self.kind = dict(kv_dtype=kv_dtype, kv_layout=kv_layout)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (NB, HKV, 1152) if kv_dtype == "e2m1" else (NB, HKV, 16, 128) if kv_layout == "hnd" else (NB, 16, HKV, 128)
        self.kc = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")  # NaN until written
        self.vc = self.kc.clone()
        self.bounds = xqa.alloc_bounds(self.kc, **self.kind)
        self.table = torch.full((PLACES, MBS), -1, dtype=torch.int32, device="cuda")
        self.lens, self.free = i32([0] * PLACES), torch.randperm(NB).to(torch.int32).cuda()
        self.num_free, self.status = i32([NB]), i32([0])

    def rows(self, n, heads):
        return torch.randn(n, heads, 128, device="cuda", generator=self.g).half()

    def grow(self, new):
        """Pages for new tokens, their keys and values and bounds; returns their offsets."""
        cu, slots, positions = xqa.xqa_assign_pages(i32(new), self.lens, self.table, self.free,
                                                    self.num_free, ROWS, status=self.status)
        k, v = self.rows(ROWS, HKV), self.rows(ROWS, HKV)
        xqa.xqa_append(k, v, cu, self.kc, self.vc, self.table, self.lens, KS, VS, status=self.status, **self.kind)
        xqa.xqa_page_bounds(self.kc, self.table, self.lens, cu, ROWS, self.bounds, status=self.status, **self.kind)
        live = sum(new)
        page = torch.repeat_interleave(torch.arange(PLACES, device="cuda"), torch.tensor(new, device="cuda"))
        assert torch.equal(slots[:live] // 16, self.table[page, (positions[:live] // 16).long()])
        assert bool((slots[live:] == -1).all())
        return cu

    def values(self, pool, scale):
        """(values of every sequence's tokens packed, their numbers)"""
        p = pool.cpu().numpy()
        if self.kind["kv_dtype"] == "e2m1":
            p = np.asarray(e2m1.decode_slices(p), np.float64)
        else:
            p = attention.code_table(self.kind["kv_dtype"]).astype(np.float64)[p]
            p = p.swapaxes(1, 2) if self.kind["kv_layout"] == "nhd" else p
        lens, table = self.lens.tolist(), self.table.cpu().numpy()
        rows = [p[table[b, :(c + 15) // 16]].swapaxes(1, 2).reshape(-1, HKV, 128)[:c] for b, c in enumerate(lens)]
        return torch.from_numpy(np.concatenate(rows)).cuda() * scale, lens

    def check_pages(self):
        lens, table = self.lens.tolist(), self.table.tolist()
        used = [table[b][j] for b in range(PLACES) for j in range((lens[b] + 15) // 16)]
        assert sorted(used + self.free[:int(self.num_free)].tolist()) == list(range(NB))
        assert int(self.status) == xqa.XQA_OK


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
def test_chunks_tokens_and_ends(kv_dtype, kv_layout):
    s = Server(kv_dtype, kv_layout, seed=len(kv_layout))
    # a prompt in chunks, others beside it: one whole prompt, single tokens, idle places
    for new in ([200, 33, 0, 0], [150, 1, 400, 0], [17, 1, 16, 5], [1, 1, 1, 1], [1, 1, 1, 1]):
        cu = s.grow(new)
        q = s.rows(ROWS, HQ)
        out = xqa.xqa_extend(q, s.kc, s.vc, s.table, s.lens, cu, KS, VS, **s.kind)
        k, lens = s.values(s.kc, KS)
        v, _ = s.values(s.vc, VS)
        n = sum(new)
        want, _, big = plain(q[:n], k, v, new, lens, True)
        compare(out[:n], want, big, torch.float16)
        s.check_pages()
    # tokens over the pages that are worth it: all of them, then a few
    for most in (MBS, 6):
        q = s.rows(PLACES, HQ)
        sel, sel_lens = xqa.xqa_select(q, s.bounds, s.table, s.lens, most, 1, 2)
        want, want_lens = plain_select(q, s.bounds, s.table.cpu().numpy(), s.lens.tolist(), HKV, most, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(sel_lens.cpu().numpy(), want_lens)
        out = xqa.xqa_decode_selected(q, s.kc, s.vc, sel, sel_lens, KS, VS, **s.kind)
        if most == MBS:
            k, lens = s.values(s.kc, KS)
            v, _ = s.values(s.vc, VS)
            dense, _, _ = plain(q, k, v, [1] * PLACES, lens, False)
            assert bool(((out.double() - dense).abs() <= ATOL + RTOL * dense.abs()).all())
        assert bool(torch.isfinite(out).all())
    # two requests end, a new one takes their place and their pages
    xqa.xqa_release_pages(torch.tensor([True, False, True, False]).cuda(), s.lens, s.table, s.free, s.num_free,
                          status=s.status)
    s.check_pages()
    cu = s.grow([0, 1, 500, 1])
    q = s.rows(ROWS, HQ)
    out = xqa.xqa_extend(q, s.kc, s.vc, s.table, s.lens, cu, KS, VS, **s.kind)
    k, lens = s.values(s.kc, KS)
    v, _ = s.values(s.vc, VS)
    want, _, big = plain(q[:502], k, v, [0, 1, 500, 1], lens, True)
    compare(out[:502], want, big, torch.float16)
    s.check_pages()


def test_a_decode_step_in_one_graph():
    """Pages, append, bounds, choice and attention of a step captured once and replayed while the
    sequences grow over page borders."""
    s = Server("e5m2", "hnd", seed=1)
    s.grow([100, 14, 260, 1])
    one, cu = i32([1] * PLACES), i32([0] * (PLACES + 1))
    slots, positions = i32([0] * PLACES), i32([0] * PLACES)
    q, k, v = s.rows(PLACES, HQ), s.rows(PLACES, HKV), s.rows(PLACES, HKV)
    shape = xqa.make_select_shape(q, s.bounds, s.table, 6, 1, 2)
    sel, lens = torch.zeros(PLACES, HKV, 6, dtype=torch.int32, device="cuda"), i32([[0] * HKV] * PLACES)
    ws = xqa.alloc_select_workspace(shape)
    dshape = xqa.make_selected_shape(q, s.kc, sel)
    dws, out = xqa.alloc_workspace(dshape), torch.zeros_like(q)

    def step():
        xqa.xqa_assign_pages(one, s.lens, s.table, s.free, s.num_free, PLACES, cu_seqlens=cu, slots=slots,
                             positions=positions, status=s.status)
        xqa.xqa_append(k, v, cu, s.kc, s.vc, s.table, s.lens, KS, VS, status=s.status)
        xqa.xqa_page_bounds(s.kc, s.table, s.lens, cu, PLACES, s.bounds, status=s.status)
        xqa.xqa_select(q, s.bounds, s.table, s.lens, selected=sel, selected_lens=lens, workspace=ws, shape=shape)
        xqa.xqa_decode_selected(q, s.kc, s.vc, sel, lens, KS, VS, out=out, workspace=dws, shape=dshape)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start = s.lens.tolist()
    for i in range(20):
        q.copy_(s.rows(PLACES, HQ))
        k.copy_(s.rows(PLACES, HKV))
        v.copy_(s.rows(PLACES, HKV))
        graph.replay()
        torch.cuda.synchronize()
        assert s.lens.tolist() == [c + i + 1 for c in start]
        assert positions.tolist() == [c + i for c in start]
        want, want_lens = plain_select(q, s.bounds, s.table.cpu().numpy(), s.lens.tolist(), HKV, 6, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(lens.cpu().numpy(), want_lens)
        fresh = xqa.xqa_decode_selected(q, s.kc, s.vc, sel, lens, KS, VS)
        assert torch.equal(fresh, out)
        s.check_pages()
    assert xqa.xqa_read_status(ws) == xqa.XQA_OK and xqa.xqa_read_status(dws) == xqa.XQA_OK

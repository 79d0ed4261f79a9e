"""One workspace for choices of different shapes in turn, and for the attention calls between
them. Choices are whole numbers: they have to equal a plain implementation."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_extend import Call, compare
from test_gpu_select import Sparse, close, plain_select, plain_selected

pytestmark = pytest.mark.gpu


def choose(s, ws, k, status=xqa.XQA_OK, **kw):
    shape = xqa.make_select_shape(s.q, s.bounds, s.c.bt, k, 1, 2, **kw)
    out = [torch.full((len(s.c.ctx), s.c.hkv, k), -5, dtype=torch.int32, device="cuda"),
           torch.full((len(s.c.ctx), s.c.hkv), -5, dtype=torch.int32, device="cuda")]
    xqa.xqa_select(s.q, s.bounds, s.c.bt, s.c.lens, selected=out[0], selected_lens=out[1],
                   workspace=ws, shape=shape)
    want = plain_select(s.q, s.bounds, s.c.table, s.c.ctx, s.c.hkv, k, 1, 2)
    for got, w in zip(out, want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert xqa.xqa_read_status(ws) == status
    return out


def test_batches_of_every_size_on_one_workspace():
    """Lengths of several chunks each, so that every segment takes a ticket; a batch's keys lie
    where the next one's did."""
    every = [Sparse([9000 + 700 * b for b in range(n)], 4, hkv, seed=n) for n, hkv in
             ((1, 1), (7, 4), (2, 4), (3, 1), (1, 4), (12, 2))]
    ws = torch.zeros(max(xqa.xqa_select_workspace_size(xqa.make_select_shape(s.q, s.bounds, s.c.bt, 40, 1, 2))
                         for s in every), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for s in every:
            choose(s, ws, 40)
            choose(s, ws, 250, max_ctas=1 + len(s.c.ctx))


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
def test_choices_and_attention_on_one_workspace(kv_dtype, kv_layout):
    s = Sparse([9000, 500, 4100], 8, 2, kv_dtype, kv_layout, seed=3)
    c = Call([40, 3, 500], [5000, 9000, 3500], seed=4, kv_dtype=kv_dtype, kv_layout=kv_layout)
    eshape = xqa.make_extend_shape(c.q, c.cache.k, c.cache.bt, **c.cache.kind)
    sel = torch.zeros((3, 2, 40), dtype=torch.int32, device="cuda")
    dshape = xqa.make_selected_shape(s.q, s.c.k, sel, **s.c.kind)
    cshape = xqa.make_select_shape(s.q, s.bounds, s.c.bt, 40, 1, 2)
    ws = torch.zeros(max(xqa.xqa_extend_workspace_size(eshape), xqa.xqa_workspace_size(dshape),
                         xqa.xqa_select_workspace_size(cshape)), dtype=torch.uint8, device="cuda")
    want, _, big = c.want()
    for _ in range(2):
        sel, lens = choose(s, ws, 40)
        out = xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, 1.0, 1.0, workspace=ws, shape=dshape)
        close(out, plain_selected(s, sel, lens, 1.0, 1.0))
        got = xqa.xqa_extend(c.q, c.cache.k, c.cache.v, c.cache.bt, c.cache.lens, c.cu, 1.0, 1.0,
                             workspace=ws, shape=eshape)
        compare(got, want, big, c.t)
        choose(s, ws, 40)


def test_two_shapes_in_graphs_that_share_a_workspace():
    a, b = Sparse([9000, 6000], 4, 2, seed=1), Sparse([12000], 4, 1, seed=2)
    shapes = [xqa.make_select_shape(s.q, s.bounds, s.c.bt, 40, 1, 2) for s in (a, b)]
    ws = torch.zeros(max(map(xqa.xqa_select_workspace_size, shapes)), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros((len(s.c.ctx), s.c.hkv, 40), dtype=torch.int32, device="cuda"),
             torch.zeros((len(s.c.ctx), s.c.hkv), dtype=torch.int32, device="cuda")) for s in (a, b)]
    graphs = []
    for s, shape, out in zip((a, b), shapes, outs):
        call = lambda: xqa.xqa_select(s.q, s.bounds, s.c.bt, s.c.lens, selected=out[0], selected_lens=out[1],
                                      workspace=ws, shape=shape)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        for x in outs[i]:
            x.fill_(-5)
        graphs[i].replay()
        s = (a, b)[i]
        for got, w in zip(outs[i], plain_select(s.q, s.bounds, s.c.table, s.c.ctx, s.c.hkv, 40, 1, 2)):
            assert np.array_equal(got.cpu().numpy(), w)

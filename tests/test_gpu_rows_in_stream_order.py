"""Calls behind one another in one stream (gather, append and gather again; decode on the rows
of the decode before): each call sees what the one before it wrote, although its threads may
be resident while earlier calls still run."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_rows import FORMATS, Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows", [[1, 2, 1], [40, 3, 17], [3000, 1, 900]])
@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
def test_each_call_sees_the_one_before(kv_dtype, kv_layout, rows, captured):
    # the same last tokens are overwritten in every step, in sectors that they share with
    # tokens the gathers before have read
    steps = 12
    ctx = [n + 60 for n in rows]
    r = Rows(rows, ctx, 2, kv_dtype, kv_layout, seed=1)
    total = sum(ctx)
    cu = torch.tensor([0, *torch.tensor(ctx).cumsum(0).tolist()], dtype=torch.int32).cuda()
    r.kc.zero_(), r.vc.zero_()
    src = [(torch.randn_like(r.k), torch.randn_like(r.v)) for _ in range(steps)]
    out = [tuple(torch.full((total, 2, 128), 5.0, dtype=torch.float16, device="cuda") for _ in range(2))
           for _ in range(2 * steps)]

    def run(outs, wait):
        for i, (k, v) in enumerate(src):
            r.gather(total, 0.5, 0.25, cu=cu, k=outs[2 * i][0], v=outs[2 * i][1])
            wait()
            r.k, r.v = k, v
            r.append(0.5, 0.25)
            wait()
            r.gather(total, 0.5, 0.25, cu=cu, k=outs[2 * i + 1][0], v=outs[2 * i + 1][1])
            wait()

    want = [tuple(torch.empty_like(x) for x in p) for p in out]
    run(want, torch.cuda.synchronize)
    r.kc.zero_(), r.vc.zero_()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(out, lambda: None)
        r.kc.zero_(), r.vc.zero_()
        g.replay()
    else:
        run(out, lambda: None)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(out, want)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), i


def test_a_row_that_was_gathered_is_appended():
    # from one cache into another and back, through the same rows
    a = Rows([500, 30], [500, 30], 2, "e4m3", "hnd", seed=2)
    a.append(0.5, 0.5)
    want = a.gather(530, 0.5, 0.5)
    b = Rows([500, 30], [500, 30], 2, "e4m3", "nhd", seed=3)
    rows = tuple(torch.zeros_like(x) for x in want)
    for i in range(20):
        x, y = (a, b) if i % 2 == 0 else (b, a)
        x.gather(530, 0.5, 0.5, k=rows[0], v=rows[1])
        y.k, y.v = rows
        y.append(0.5, 0.5)
    b.gather(530, 0.5, 0.5, k=rows[0], v=rows[1])
    assert torch.equal(rows[0], want[0]) and torch.equal(rows[1], want[1])


@pytest.mark.parametrize("kv_dtype", ["e5m2", "e2m1"])
@pytest.mark.parametrize("ctx", [[20], [300, 17, 1000]])
def test_decode_reads_the_rows_of_the_decode_before(ctx, kv_dtype):
    r = Rows(ctx, ctx, 2, kv_dtype, "hnd", seed=4)
    r.append()
    q = torch.randn(len(ctx), 8, 128, device="cuda").half()
    shape = xqa.make_shape(q, r.kc, r.bt, kv_dtype=kv_dtype)
    ws = xqa.alloc_workspace(shape)

    def run(wait):
        a, b = q.clone(), torch.empty_like(q)
        for _ in range(10):
            xqa.xqa_decode(a, r.kc, r.vc, r.bt, r.lens, 1.0, 1.0, out=b, workspace=ws, shape=shape)
            wait()
            a, b = b, a
        torch.cuda.synchronize()
        return a

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        assert torch.equal(run(lambda: None), want)

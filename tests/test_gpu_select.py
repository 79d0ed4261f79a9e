"""xqa_page_bounds, xqa_select and xqa_decode_selected.

Bounds and choices are whole numbers: they have to equal a plain implementation in 64 bits.
Attention over the selected pages is held against float64 softmax over their values, with
the tolerance of decode (gpu_helpers.py).
"""
import math

import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from gpu_helpers import ATOL, RTOL
from test_gpu_extend import FORMATS, Cache, i32
from test_gpu_prefill import offsets

pytestmark = pytest.mark.gpu


def page_values(cache, pool):
    """[NB, Hkv, 16, 128] in 64 bits, before the scale."""
    from oracle import attention, e2m1

    p = pool.cpu().numpy()
    if cache.kv_dtype == "e2m1":
        return np.asarray(e2m1.decode_slices(p), np.float64)
    p = attention.code_table(cache.kv_dtype).astype(np.float64)[p]
    return p.swapaxes(1, 2) if cache.kv_layout == "nhd" else p


def plain_bounds(cache, before, new, ctx):
    res = before.cpu().numpy().copy().view(np.int8)
    x = page_values(cache, cache.k)
    for b, (n, c) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        for j in range((c - n) // 16, (c + 15) // 16):
            page = cache.table[b, j]
            for h in range(cache.hkv):
                k = x[page, h, :min(16, c - 16 * j)]
                row = np.zeros(272, np.float64)
                top = np.abs(k).max()
                if not np.isfinite(k).all():
                    row[256] = -128
                elif top > 0:
                    e = math.floor(math.log2(top)) - 6
                    assert 64 <= top / 2.0**e < 128
                    row[:128], row[128:256], row[256] = np.ceil(k.max(0) / 2.0**e), np.floor(k.min(0) / 2.0**e), e
                res[page, h] = row.astype(np.int8)
    return res


def bounds_of(cache, new, **kw):
    bounds = xqa.alloc_bounds(cache.k, **cache.kind)
    bounds.fill_(77)
    before = bounds.clone()
    status = i32([0])
    xqa.xqa_page_bounds(cache.k, cache.bt, cache.lens, offsets(new), sum(new) + kw.pop("pad", 0), bounds,
                        status=status, **cache.kind)
    assert int(status) == kw.pop("status", 0)
    return bounds, before


@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
@pytest.mark.parametrize("new,ctx", [([1], [1]), ([1, 1, 1], [16, 17, 300]), ([5, 0, 40, 16], [5, 9, 100, 33]),
                                     ([200, 3], [200, 1000])])
def test_bounds(new, ctx, kv_dtype, kv_layout):
    c = Cache(ctx, 3, kv_dtype, kv_layout, seed=sum(ctx))
    got, before = bounds_of(c, new, pad=3)
    assert np.array_equal(got.cpu().numpy().view(np.int8), plain_bounds(c, before, new, ctx))


def test_bounds_of_many_rows():
    new = [2100, 1, 1900, 700]  # more than 4096 rows: a warp takes more of them
    ctx = [2100, 2000, 1907, 715]
    c = Cache(ctx, 2, "e4m3", "nhd", seed=1)
    got, before = bounds_of(c, new)
    assert np.array_equal(got.cpu().numpy().view(np.int8), plain_bounds(c, before, new, ctx))


@pytest.mark.parametrize("kv_dtype", ["e5m2", "e4m3", "e2m1"])
def test_bounds_hold_every_key_of_any_codes(kv_dtype):
    """Random codes over the whole range of the format, zeros, smallest and largest values."""
    g = np.random.default_rng(3)
    c = Cache([16] * 40, 2, kv_dtype, "hnd", seed=1)
    raw = g.integers(0, 256, c.k.shape).astype(np.uint8)
    if kv_dtype == "e2m1":
        raw[:, :, 1024:][raw[:, :, 1024:] % 128 == 127] = 1
        raw[c.table[0, 0]] = 0
        raw[c.table[1, 0], :, 1024:] = 1      # the smallest scale
        raw[c.table[2, 0], :, 1024:] = 0x7E   # the largest
    else:
        limit = 0x7C if kv_dtype == "e5m2" else 0x7F
        raw[raw % 128 >= limit] = 0
        raw[c.table[0, 0]] = 0x80             # zeros of either sign
        raw[c.table[1, 0]] = g.integers(0, 2, raw[0].shape)
        raw[c.table[2, 0]] = limit - 1
    c.k.copy_(torch.from_numpy(raw))
    new = [16] * 40
    got, before = bounds_of(c, new)
    want = plain_bounds(c, before, new, c.ctx)
    got = got.cpu().numpy().view(np.int8)
    assert np.array_equal(got, want)
    x = page_values(c, c.k)
    for b in range(40):
        page = c.table[b, 0]
        scale = 2.0 ** got[page, :, 256:257].astype(np.float64)
        assert (got[page, :, :128] * scale >= x[page].max(1)).all()
        assert (got[page, :, 128:256] * scale <= x[page].min(1)).all()


@pytest.mark.parametrize("kv_dtype,bad", [("e5m2", 0x7C), ("e5m2", 0xFF), ("e4m3", 0xFF)])
def test_bounds_of_keys_that_are_not_finite(kv_dtype, bad):
    c = Cache([40, 20], 2, kv_dtype, "hnd", seed=1)
    c.slot("k", 0, 17, 1)[3] = bad
    got, before = bounds_of(c, [40, 20])
    assert np.array_equal(got.cpu().numpy().view(np.int8), plain_bounds(c, before, [40, 20], c.ctx))
    assert int(got.view(torch.int8)[int(c.table[0, 1]), 1, 256]) == -128


def test_bounds_errors():
    c = Cache([40, 20, 50], 2, "e5m2", "hnd", seed=1, mbs=8)
    good, _ = bounds_of(c, [40, 20, 1])
    c.bt[0, 1] = c.nb
    got, before = bounds_of(c, [40, 20, 1], status=xqa.XQA_ERR_BAD_BLOCK_ID)
    page = int(c.table[0, 1])
    good[page] = before[page]
    assert torch.equal(got, good)
    for length in (-1, 19, 129):
        c = Cache([40, 20, 50], 2, "e5m2", "hnd", seed=1, mbs=8)
        good, _ = bounds_of(c, [40, 20, 1])
        c.lens[1] = length
        got, before = bounds_of(c, [40, 20, 1], status=xqa.XQA_ERR_CTX_TOO_LONG)
        for page in c.table[1, :2]:
            good[int(page)] = before[int(page)]
        assert torch.equal(got, good)


# ---- the choice ----
def plain_select(q, bounds, table, ctx, hkv, k, first, last):
    b, hq = q.shape[:2]
    g = hq // hkv
    bd = bounds.cpu().numpy().view(np.int8).astype(np.float64)
    qn = q.cpu().numpy().astype(np.float64)
    selected, lens = np.full((b, hkv, k), -1, np.int32), np.zeros((b, hkv), np.int32)
    for i, c in enumerate(ctx):
        num = (c + 15) // 16
        for h in range(hkv):
            x = np.where(np.isfinite(qn[i, h * g:(h + 1) * g]), qn[i, h * g:(h + 1) * g], 0)
            top = np.abs(x).max()
            f = math.floor(math.log2(top)) - 5 if top > 0 else 0
            w = np.rint(x / 2.0**f)
            rows = bd[table[i, :num], h]
            score = (rows[:, :128] @ np.maximum(w, 0).sum(0) + rows[:, 128:256] @ np.minimum(w, 0).sum(0)) \
                * 2.0 ** rows[:, 256]
            score = np.where(rows[:, 256] == -128, np.inf, score)
            always = [j for j in range(num) if j < first or j >= num - last]
            rest = sorted((j for j in range(num) if j not in set(always)), key=lambda j: (-score[j], j))
            take = sorted((always + rest)[:k]) if num > k else list(range(num))
            selected[i, h, :len(take)] = table[i, take]
            lens[i, h] = c - (num - len(take)) * 16
    return selected, lens


class Sparse:
    def __init__(self, ctx, hq=8, hkv=2, kv_dtype="e5m2", kv_layout="hnd", seed=0, mbs=None):
        self.c = Cache(ctx, hkv, kv_dtype, kv_layout, seed, mbs=mbs)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q = torch.randn(len(ctx), hq, 128, device="cuda", generator=g).half()
        self.bounds = xqa.alloc_bounds(self.c.k, **self.c.kind)
        if sum(ctx):
            xqa.xqa_page_bounds(self.c.k, self.c.bt, self.c.lens, offsets(ctx), sum(ctx), self.bounds,
                                **self.c.kind)

    def choose(self, k, first=1, last=1, status=xqa.XQA_OK, **kw):
        shape = xqa.make_select_shape(self.q, self.bounds, self.c.bt, k, first, last, **kw)
        ws = xqa.alloc_select_workspace(shape)
        for _ in range(2):  # the workspace is left ready
            sel, lens = xqa.xqa_select(self.q, self.bounds, self.c.bt, self.c.lens, workspace=ws, shape=shape)
        torch.cuda.synchronize()
        assert xqa.xqa_read_status(ws) == status
        return sel, lens

    def check(self, k, first=1, last=1, **kw):
        sel, lens = self.choose(k, first, last, **kw)
        want, wlens = plain_select(self.q, self.bounds, self.c.table, self.c.ctx, self.c.hkv, k, first, last)
        assert np.array_equal(lens.cpu().numpy(), wlens)
        assert np.array_equal(sel.cpu().numpy(), want)
        return sel, lens


@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
def test_choices(kv_dtype, kv_layout):
    s = Sparse([1, 16, 17, 0, 500, 1000, 159, 160, 161], kv_dtype=kv_dtype, kv_layout=kv_layout, seed=2)
    for k, first, last in ((10, 1, 1), (1, 0, 1), (2, 1, 1), (33, 4, 16), (100, 0, 2)):
        s.check(k, first, last)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 1), (7, 1), (12, 4), (16, 16)])
def test_choices_of_head_groups(hq, hkv):
    Sparse([800, 333], hq, hkv, seed=hq).check(12, 2, 3)


@pytest.mark.parametrize("max_ctas", [1, 5, 0])
@pytest.mark.parametrize("ctx", [[9000, 20, 4100], [16 * 257, 16 * 256, 16 * 255]])
def test_choices_in_chunks(ctx, max_ctas):
    s = Sparse(ctx, 4, 2, seed=5)
    s.check(40, 1, 2, max_ctas=max_ctas)
    s.check(250, 0, 1, max_ctas=max_ctas)


def test_ties_go_to_the_lower_page():
    s = Sparse([2000], 4, 1, seed=1)
    s.bounds[:, :, :128], s.bounds[:, :, 128:256], s.bounds[:, :, 256] = 5, 250, 0  # all pages alike
    s.check(17, 1, 2)
    s.bounds[s.c.table[0, 60]] = 0  # one lower than the others
    s.check(123, 1, 1)
    s.q.zero_()
    s.check(17, 1, 2)


def test_ties_over_the_longest_table():
    # every lane of the CTA that chooses counts 2^15 equal keys
    mbs, nb = 1 << 24, 7
    bounds = torch.zeros((nb, 1, 272), dtype=torch.uint8, device="cuda")
    table = (torch.arange(mbs, device="cuda") % nb).to(torch.int32).reshape(1, mbs)
    q = torch.ones((1, 1, 128), dtype=torch.float16, device="cuda")
    selected, lens = xqa.xqa_select(q, bounds, table, i32([16 * mbs]), 6, 1, 2)
    assert selected[0, 0].tolist() == [0, 1, 2, 3, (mbs - 2) % nb, (mbs - 1) % nb]
    assert lens.tolist() == [[96]]


def test_large_and_odd_queries_and_bounds():
    s = Sparse([1500, 700], 16, 1, seed=1)
    s.q.fill_(65504.0)
    s.bounds.view(torch.int8)[:, :, :128] = 127  # the largest sums there can be
    s.check(20)
    s.q.copy_(torch.randn_like(s.q) * 2.0**-24 * 40)  # subnormal numbers
    s.check(20)
    s.q[0, 3, 5], s.q[0, 2, 9], s.q[1, 0, 0] = math.inf, math.nan, -math.inf
    s.check(20)
    s.c.slot("k", 0, 33, 0)[4] = 0x7F
    xqa.xqa_page_bounds(s.c.k, s.c.bt, s.c.lens, offsets([1500, 700]), 2200, s.bounds)
    sel, _ = s.check(20)
    assert int(s.c.table[0, 2]) in sel[0, 0].tolist()


def test_choice_errors():
    s = Sparse([1500, 700, 90], 4, 2, seed=1, mbs=100)
    want, wlens = s.choose(20)
    s.c.bt[0, 50] = -3
    sel, lens = s.choose(20, status=xqa.XQA_ERR_BAD_BLOCK_ID)
    assert bool((sel[0] == -3).any(dim=1).all()) and torch.equal(sel[1:], want[1:])
    s.c.bt[0, 50] = int(s.c.table[0, 50])
    for length in (-1, 1601):
        s.c.lens[1] = length
        sel, lens = s.choose(20, status=xqa.XQA_ERR_CTX_TOO_LONG)
        assert bool((sel[1] == -1).all()) and bool((lens[1] == -1).all())
        assert torch.equal(sel[0], want[0]) and torch.equal(lens[2], wlens[2])


# ---- attention over the choice ----
def plain_selected(s, sel, lens, ks, vs):
    g = s.q.shape[1] // s.c.hkv
    k, v = (page_values(s.c, p) for p in (s.c.k, s.c.v))
    out = np.zeros(s.q.shape)
    for b in range(s.q.shape[0]):
        for h in range(s.c.hkv):
            n = int(lens[b, h])
            if n == 0:
                continue
            pages = sel[b, h, :(n + 15) // 16].tolist()
            kk, vv = (x[pages, h].reshape(-1, 128)[:n] for x in (k, v))
            q = s.q[b, h * g:(h + 1) * g].double().cpu().numpy()
            z = q @ kk.T * ks / math.sqrt(128)
            w = np.exp(z - z.max(1, keepdims=True))
            out[b, h * g:(h + 1) * g] = w @ vv / w.sum(1, keepdims=True) * vs
    return out


def close(got, want):
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= ATOL + RTOL * np.abs(want)).all(), float(err.max())


@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
@pytest.mark.parametrize("ctx,hq,hkv,k", [([500, 1000, 3, 0, 161], 8, 2, 12), ([3000], 16, 1, 40), ([700] * 5, 12, 4, 9),
                                          ([70, 200] * 170, 8, 4, 3)])
def test_attention_over_selected_pages(ctx, hq, hkv, k, kv_dtype, kv_layout):
    s = Sparse(ctx, hq, hkv, kv_dtype, kv_layout, seed=k)
    sel, lens = s.check(k, 1, 1)
    shape = xqa.make_selected_shape(s.q, s.c.k, sel, **s.c.kind)
    ws = xqa.alloc_workspace(shape)
    for _ in range(2):
        out = xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, 0.5, 0.25, workspace=ws, shape=shape)
    assert xqa.xqa_read_status(ws) == xqa.XQA_OK
    close(out, plain_selected(s, sel, lens, 0.5, 0.25))
    dev = [torch.tensor([x], device="cuda") for x in (0.5, 0.25)]
    again = xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, *dev, workspace=ws, shape=shape)
    assert torch.equal(again, out)


@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
def test_all_pages_are_dense_attention(kv_dtype, kv_layout):
    s = Sparse([500, 1000, 3], 8, 2, kv_dtype, kv_layout, seed=3)
    sel, lens = s.choose(70)
    out = xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, 1.0, 1.0, **s.c.kind)
    dense = xqa.xqa_decode(s.q, s.c.k, s.c.v, s.c.bt, s.c.lens, 1.0, 1.0, **s.c.kind)
    # the same pages, cut elsewhere: each is within 2^-11 of the largest value or so
    assert bool(((out.float() - dense.float()).abs() <= ATOL + RTOL * dense.float().abs()).all())


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "nhd"), ("e4m3", "hnd")])
def test_a_batch_that_needs_the_planner_and_the_combine_kernel(kv_dtype, kv_layout):
    s = Sparse([40, 100, 70] * 180, 8, 4, kv_dtype, kv_layout, seed=3)  # 2160 segments
    sel, lens = s.choose(3, 0, 1)
    want = plain_selected(s, sel, lens, 1.0, 1.0)
    for mode in (0, 1):
        shape = xqa.make_selected_shape(s.q, s.c.k, sel, merge_mode=mode, **s.c.kind)
        close(xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, 1.0, 1.0, shape=shape), want)


def test_errors_that_the_choice_passes_on():
    s = Sparse([1500, 700, 90], 4, 2, seed=1, mbs=100)
    s.c.bt[0, 50] = -3
    s.c.lens[1] = -1
    sel, lens = xqa.xqa_select(s.q, s.bounds, s.c.bt, s.c.lens, 20)
    shape = xqa.make_selected_shape(s.q, s.c.k, sel)
    ws = xqa.alloc_workspace(shape)
    out = xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, 1.0, 1.0, workspace=ws, shape=shape)
    assert xqa.xqa_read_status(ws) in (xqa.XQA_ERR_BAD_BLOCK_ID, xqa.XQA_ERR_CTX_TOO_LONG)
    assert bool(torch.isnan(out[:2]).all()) and bool(torch.isfinite(out[2]).all())


def test_graph_streams_and_two_calls_at_once():
    a, b = Sparse([3000, 800], seed=1), Sparse([900] * 9, kv_dtype="e4m3", kv_layout="nhd", seed=2)

    def step(s, stream=None):
        sel, lens = xqa.xqa_select(s.q, s.bounds, s.c.bt, s.c.lens, 16, 1, 2, stream=stream)
        return sel, xqa.xqa_decode_selected(s.q, s.c.k, s.c.v, sel, lens, 1.0, 1.0, stream=stream, **s.c.kind)

    want = [step(a), step(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [step(s, t) for s, t in zip((a, b), streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    shape = xqa.make_select_shape(a.q, a.bounds, a.c.bt, 16, 1, 2)
    sel, lens = torch.zeros(2, 2, 16, dtype=torch.int32, device="cuda"), i32([[0, 0], [0, 0]])
    ws, dshape = xqa.alloc_select_workspace(shape), xqa.make_selected_shape(a.q, a.c.k, sel)
    dws, out = xqa.alloc_workspace(dshape), torch.zeros_like(a.q)
    graph = torch.cuda.CUDAGraph()

    def call():
        xqa.xqa_select(a.q, a.bounds, a.c.bt, a.c.lens, selected=sel, selected_lens=lens, workspace=ws,
                       shape=shape)
        xqa.xqa_decode_selected(a.q, a.c.k, a.c.v, sel, lens, 1.0, 1.0, out=out, workspace=dws, shape=dshape)

    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    assert torch.equal(out, want[0][1])
    a.q.copy_(a.q.flip(1))
    graph.replay()
    got = out.clone()
    s2, o2 = step(a)
    assert torch.equal(sel, s2) and torch.equal(got, o2)


def test_binding_refusals():
    s = Sparse([300, 90], seed=1)
    c = s.c
    for args, kw in (((s.q.float(), s.bounds, c.bt, c.lens, 8), {}), ((s.q, s.bounds[:, :, :16], c.bt, c.lens, 8), {}),
                     ((s.q, s.bounds, c.bt.long(), c.lens, 8), {}), ((s.q, s.bounds, c.bt, c.lens[:1], 8), {}),
                     ((s.q, s.bounds, c.bt, c.lens, 0), {}), ((s.q, s.bounds, c.bt, c.lens, 4, 3, 2), {}),
                     ((s.q, s.bounds, c.bt, c.lens, 4, 3, 0), {}), ((s.q, s.bounds, c.bt, c.lens, 4, -1, 1), {}),
                     ((s.q.cpu(), s.bounds, c.bt, c.lens, 8), {}), ((s.q[:1], s.bounds, c.bt, c.lens, 8), {}),
                     ((s.q, s.bounds, c.bt, c.lens, 8), dict(selected=i32([[1]]))),
                     ((s.q, s.bounds, c.bt, c.lens, 8), dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")))):
        with pytest.raises((ValueError, xqa.XqaError)):
            xqa.xqa_select(*args, **kw)
    sel, lens = s.choose(8)
    for args in ((s.q, c.k, c.v, sel[:, :1], lens, 1.0, 1.0), (s.q, c.k, c.v, sel, lens[:, :1], 1.0, 1.0),
                 (s.q, c.k, c.v, sel.long(), lens, 1.0, 1.0), (s.q[:, None], c.k, c.v, sel, lens, 1.0, 1.0),
                 (s.q, c.k, c.v[:1], sel, lens, 1.0, 1.0), (s.q, c.k, c.v, sel, lens, torch.ones(1, device="cuda"), 1.0)):
        with pytest.raises((ValueError, xqa.XqaError)):
            xqa.xqa_decode_selected(*args)
    cu = offsets([300, 90])
    for bad in ((c.k.cpu(), c.bt, c.lens, cu, 390, s.bounds), (c.k, c.bt, c.lens, cu[:2], 390, s.bounds),
                (c.k, c.bt, c.lens, cu, 390, s.bounds[:1]), (c.k, c.bt, c.lens, cu, -1, s.bounds),
                (c.k, c.bt.float(), c.lens, cu, 390, s.bounds)):
        with pytest.raises((ValueError, xqa.XqaError)):
            xqa.xqa_page_bounds(*bad)

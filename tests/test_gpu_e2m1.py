"""Decode over the 4-bit cache against the float64 oracle, through every entry point.

Tolerance: dequantisation is exact (s * code has at most 6 significant bits and
is an fp16 value), logits are 32-bit sums of exact products. The fp16 weights are
off by at most u = 2^-11 each and their sum takes the rounded ones, so the row
moves by at most u * sum_j w_j |v_j - out| <= u (max |v| + |out|); the output is
rounded once more: |got - out| <= 1.05 u (max |v| + 2 |out|) + 1e-6.
"""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from gpu_helpers import to_dev
from oracle import e2m1, e4m3

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, ctx, hq, hkv, q_len=1, seed=0, ks=1.0, vs=1.0, big=False):
        rng = np.random.default_rng(seed)
        self.ctx, self.hq, self.hkv, self.ks, self.vs = list(ctx), hq, hkv, ks, vs
        pages = [(max(0, c) + 15) // 16 for c in self.ctx]
        self.nb, self.mbs = sum(pages) + 5, max(1, max(pages))
        order = rng.permutation(self.nb)
        self.table = np.full((len(self.ctx), self.mbs), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        # random codes; scales over a few binades (over all finite ones with `big`); what lies
        # behind a sequence, and unused pages, keep NaN scales
        self.cache = []
        for _ in range(2):
            c = rng.integers(0, 256, (self.nb, hkv, 1152), dtype=np.uint8)
            sc = c[:, :, 1024:].reshape(self.nb, hkv, 16, 8)
            sc[:] = rng.integers(0, 127, sc.shape) if big else rng.integers(0x28, 0x38, sc.shape)
            used = np.zeros((self.nb, 16), bool)
            for b, n in enumerate(self.ctx):
                pos = np.arange(max(0, n))
                used[self.table[b, pos // 16], pos % 16] = True
            sc[~used.repeat(hkv, 0).reshape(self.nb, hkv, 16)] = 0x7F
            self.cache.append(c)
        shape = (len(self.ctx), hq, 128) if q_len == 1 else (len(self.ctx), q_len, hq, 128)
        self.q = rng.standard_normal(shape).astype(np.float16)

    def dev(self, **kw):
        return Dev(self, **kw)

    def oracle(self, sm_scale=None):
        return e2m1.paged_decode_attention(self.q, self.cache[0], self.cache[1], self.table,
                                           [max(0, c) for c in self.ctx], self.ks, self.vs, sm_scale)

    def check(self, got, sm_scale=None, rows=None):
        want = self.oracle(sm_scale)
        got = got.astype(np.float64)
        vmax = np.zeros(len(self.ctx))
        for b, n in enumerate(self.ctx):
            pages = self.table[b, :(max(0, n) + 15) // 16]
            v = e2m1.decode_slices(self.cache[1][pages]).swapaxes(1, 2).reshape(-1, self.hkv, 128)[:max(0, n)]
            vmax[b] = np.abs(v).max() * self.vs if n > 0 else 0
        if rows is not None:
            want, got, vmax = want[rows], got[rows], vmax[rows]
        u = 2.0**-11
        bound = 1.05 * u * (vmax.reshape(-1, *[1] * (want.ndim - 1)) + 2 * np.abs(want)) + 1e-6
        bad = ~(np.abs(got - want) <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], want[bad][0])


class Dev:
    def __init__(self, c, merge_mode=0, max_ctas=0, min_pages=0, sm_scale=0.0):
        self.c = c
        self.q, self.bt = to_dev(c.q), to_dev(c.table)
        self.k, self.v = (to_dev(x) for x in c.cache)
        self.lens = torch.tensor(c.ctx, dtype=torch.int32).cuda()
        self.shape = xqa.make_shape(self.q, self.k, self.bt, sm_scale, max_ctas, min_pages, merge_mode,
                                    kv_dtype="e2m1")
        self.ws = xqa.alloc_workspace(self.shape)
        self.out = torch.full_like(self.q, float("nan"))

    def run(self, ok=True):
        xqa.xqa_decode(self.q, self.k, self.v, self.bt, self.lens, self.c.ks, self.c.vs, out=self.out,
                       workspace=self.ws, shape=self.shape)
        torch.cuda.synchronize()
        if ok:
            assert xqa.xqa_read_status(self.ws) == xqa.XQA_OK
        assert not bool(self.ws[64:64 + 8 * 1024].any())  # merge tickets at zero
        return self.out.cpu().numpy()


@pytest.mark.parametrize("merge_mode", [0, 1])
@pytest.mark.parametrize("ctx", [[1], [16], [17], [256], [1, 15, 16, 17, 33], [0, 5, 0, 64], [1000, 300]])
def test_small_contexts(ctx, merge_mode):
    c = Case(ctx, 8, 1, seed=len(ctx))
    c.check(c.dev(merge_mode=merge_mode).run())


@pytest.mark.parametrize("hq,hkv", [(4, 4), (16, 4), (24, 3), (2, 2), (32, 2), (16, 1), (7, 1), (32, 4)])
def test_group_sizes(hq, hkv):
    c = Case([1, 16, 17, 300, 2049], hq, hkv, seed=hq, ks=0.5, vs=0.25)
    c.check(c.dev().run())


@pytest.mark.parametrize("q_len,hq,hkv", [(2, 8, 1), (2, 16, 4), (4, 8, 2), (16, 1, 1), (3, 10, 2)])
def test_new_tokens(q_len, hq, hkv):
    c = Case([q_len, 1, 40, 16, 1025], hq, hkv, q_len, seed=q_len)
    c.check(c.dev().run())
    assert np.array_equal(c.dev(merge_mode=1).run(), c.dev().run())


def test_every_scale_and_code():
    # all finite group scales, 2^-9 .. 448, on values and keys; small q keeps the softmax mixed
    c = Case([700, 64], 8, 2, seed=3, big=True, vs=2.0**-8)
    c.q = (c.q * 2.0**-9).astype(np.float16)
    c.check(c.dev().run())


@pytest.mark.parametrize("max_ctas,min_pages", [(1, 0), (7, 1), (37, 3), (0, 1), (300, 1)])
def test_splits_and_merges(max_ctas, min_pages):
    c = Case([1, 15, 4097, 16, 9000, 33], 8, 2, seed=4)
    a = c.dev(max_ctas=max_ctas, min_pages=min_pages).run()
    b = c.dev(max_ctas=max_ctas, min_pages=min_pages, merge_mode=1).run()
    assert np.array_equal(a.view(np.uint16), b.view(np.uint16))
    c.check(a)


@pytest.mark.parametrize("q_len", [1, 2])
def test_one_long_sequence(q_len):
    c = Case([70001], 16, 2, q_len, seed=5)
    c.check(c.dev().run())


@pytest.mark.parametrize("q_len", [1, 2])
def test_many_short_sequences(q_len):
    # enough segments per CTA for the warp-per-piece mode
    rng = np.random.default_rng(6)
    ctx = rng.integers(q_len, 400, 170)
    ctx[::17], ctx[5::23] = 16, q_len
    c = Case(ctx, 16, 4, q_len, seed=6)
    a = c.dev().run()
    c.check(a)
    assert np.array_equal(a, c.dev(merge_mode=1).run())


def test_more_segments_than_the_shared_table():
    rng = np.random.default_rng(7)
    ctx = rng.integers(0, 90, 600)
    c = Case(ctx, 8, 4, seed=7)
    c.check(c.dev().run())
    c.check(c.dev(max_ctas=1).run())


def test_pages_may_move_and_what_lies_behind_is_not_read():
    c = Case([33, 500, 16], 8, 2, seed=8)
    a = c.dev().run()
    rng = np.random.default_rng(9)
    perm = rng.permutation(c.nb)
    m = Case([33, 500, 16], 8, 2, seed=8)
    for x, y in zip(m.cache, c.cache):
        x[perm] = y
        codes = x[:, :, :1024].reshape(c.nb, 2, 16, 64)
        sc = x[:, :, 1024:].reshape(c.nb, 2, 16, 8)
        hidden = sc == 0x7F                      # other garbage behind the sequences
        sc[hidden] = rng.integers(0, 256, int(hidden.sum()))
        codes[hidden.any(-1)] = 0x77
    m.table = np.where(c.table >= 0, perm[c.table], 2**30).astype(np.int32)
    assert np.array_equal(a.view(np.uint16), m.dev().run().view(np.uint16))


def test_bad_pages_and_lengths_give_nan_rows():
    for mode in (0, 1):
        c = Case([40, 3000, 5000, 70, 16], 8, 2, seed=10)
        d = c.dev(merge_mode=mode)
        d.bt[1, 9] = c.nb + 2
        d.lens[3] = c.mbs * 16 + 1
        out = d.run(ok=False)
        assert xqa.xqa_read_status(d.ws) in (xqa.XQA_ERR_BAD_BLOCK_ID, xqa.XQA_ERR_CTX_TOO_LONG)
        assert np.isnan(out[[1, 3]].astype(np.float32)).all()
        c.check(out, rows=[0, 2, 4])
        d.bt.copy_(to_dev(c.table))
        d.lens.copy_(torch.tensor(c.ctx, dtype=torch.int32))
        c.check(d.run())


def test_garbage_hints_change_nothing():
    c = Case([3000, 100], 8, 2, seed=11)
    d = c.dev()
    want = d.run().copy()
    words = d.ws[64 + 12 * 1024:64 + 12 * 1024 + 4 * 16 * 1024].view(torch.int32)
    assert int((words > 0).sum()) > 0
    for fill in (2**31 - 1, -1, -2**31, 16 * c.nb * 2, 16 * c.nb * 2 - 1):
        words.fill_(fill)
        assert np.array_equal(d.run().view(np.uint16), want.view(np.uint16))


def test_other_entry_points():
    c = Case([900, 17, 1, 4100], 16, 2, seed=12, ks=0.5, vs=0.25)
    d = c.dev()
    want = d.run().copy()
    c.check(want)
    got = xqa.xqa_decode_static_workspace(d.q, d.k, d.v, d.bt, d.lens, 0.5, 0.25, kv_dtype="e2m1")
    assert np.array_equal(got.cpu().numpy(), want)
    ks, vs = torch.tensor([0.5], device="cuda"), torch.tensor([0.25], device="cuda")
    got = xqa.xqa_decode(d.q, d.k, d.v, d.bt, d.lens, ks, vs, kv_dtype="e2m1")
    assert np.array_equal(got.cpu().numpy(), want)
    s = c.dev(merge_mode=1)
    xqa.xqa_plan(s.lens, s.ws, s.shape)
    xqa.xqa_attend_partial(s.q, s.k, s.v, s.bt, s.lens, 0.5, 0.25, s.out, s.ws, s.shape)
    xqa.xqa_combine(s.lens, 0.25, s.out, s.ws, s.shape)
    torch.cuda.synchronize()
    assert np.array_equal(s.out.cpu().numpy(), want)
    a = c.dev(sm_scale=0.02).run()
    c.check(a, sm_scale=0.02)
    # captured, replayed with other lengths and other pages of q
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xqa.xqa_decode(d.q, d.k, d.v, d.bt, d.lens, 0.5, 0.25, out=d.out, workspace=d.ws, shape=d.shape)
    c.ctx = [800, 16, 1, 4099]
    d.lens.copy_(torch.tensor(c.ctx, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    c.check(d.out.cpu().numpy())


def test_nan_scale_of_a_visible_token_reaches_its_rows_only():
    c = Case([100, 100], 8, 2, seed=13)
    want = c.dev().run().copy()
    page, slot = c.table[0, 50 // 16], 50 % 16
    c.cache[1][page, 1, 1024 + slot * 8 + 3] = 0x7F
    out = c.dev().run()
    nan = np.isnan(out.astype(np.float32))
    assert nan[0, 4:, 48:64].all() and nan.sum() == 4 * 16
    assert np.array_equal(out[~nan], want[~nan])


def test_nan_scale_of_a_new_token_stays_hidden_from_those_before_it():
    for ctx in (100, 97, 16, 4):
        c = Case([ctx, 40], 8, 2, q_len=4, seed=14)
        want = c.dev().run().copy()
        for new in range(4):
            d = Case([ctx, 40], 8, 2, q_len=4, seed=14)
            at = ctx - 4 + new
            for cache in (0, 1):  # its key, then its value
                d.cache[cache][d.table[0, at // 16], 1, 1024 + at % 16 * 8 + 3] = 0x7F
                out = d.dev().run()
                nan = np.isnan(out.astype(np.float32))
                dims = slice(48, 64) if cache == 1 else slice(None)
                assert nan[0, new:, 4:, dims].all()
                assert nan.sum() == (4 - new) * 4 * (16 if cache == 1 else 128)
                nan[0, new:, 4:] = True
                assert np.array_equal(out[~nan], want[~nan])
                d.cache[cache][:] = c.cache[cache]


def test_token_major_layout_is_refused():
    c = Case([16], 8, 1)
    d = c.dev()
    d.shape.kv_layout = 1
    with pytest.raises(xqa.XqaError):
        d.run()
    with pytest.raises(ValueError):
        xqa.make_shape(d.q, d.k, d.bt, kv_dtype="e2m1", kv_layout="nhd")

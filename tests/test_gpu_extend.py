"""xqa_extend against a plain float64 implementation over the values that the cache holds.

Tolerances are those of prompt attention (test_gpu_prefill.py): weights rounded once to the
type, out rounded once, 32-bit sums. The tensor's scales are applied in 32 bits (2^-24
relative each), which the factor 1.05 covers. Every slot of the pool that no token uses holds
NaN codes.
"""
import math

import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from oracle import attention, e2m1
from test_gpu_prefill import TYPES, compare, offsets, plain

pytestmark = pytest.mark.gpu

FORMATS = [("e5m2", "hnd"), ("e5m2", "nhd"), ("e4m3", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")]


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Cache:
    """A paged cache of ``ctx`` tokens for each sequence: codes of normal values, and what
    they stand for. Slots that no token has, and pages that no sequence has, hold NaN."""

    def __init__(self, ctx, hkv, kv_dtype, kv_layout, seed=0, spread=1.0, mbs=None):
        self.ctx, self.hkv, self.kv_dtype, self.kv_layout = ctx, hkv, kv_dtype, kv_layout
        g = np.random.default_rng(seed)
        pages = [(max(c, 0) + 15) // 16 for c in ctx]
        self.mbs = mbs or max(1, max(pages))
        self.nb = sum(pages) + 5
        ids = g.permutation(self.nb).astype(np.int32)
        self.table = np.full((len(ctx), self.mbs), -7, np.int32)
        at = 0
        for b, p in enumerate(pages):
            self.table[b, :p] = ids[at:at + p]
            at += p
        self.k, self.v = (self._pool(g, spread) for _ in range(2))
        self.bt, self.lens = torch.from_numpy(self.table).cuda(), i32(ctx)

    def _pool(self, g, spread):
        used = np.zeros((self.nb, 16), bool)
        for b, c in enumerate(self.ctx):
            for t in range(max(c, 0)):
                used[self.table[b, t // 16], t % 16] = True
        x = (g.standard_normal((self.nb, self.hkv, 16, 128)) * spread).astype(np.float32)
        if self.kv_dtype == "e2m1":
            codes, scales = e2m1.encode(x, 1.0)
            scales = np.where(used[:, None, :, None], scales, 0x7F).astype(np.uint8)
            return torch.from_numpy(e2m1.pack(codes, scales)).cuda()
        t = torch.float8_e5m2 if self.kv_dtype == "e5m2" else torch.float8_e4m3fn
        codes = torch.from_numpy(x).to(t).view(torch.uint8)
        codes = torch.where(torch.from_numpy(used)[:, None, :, None], codes, torch.tensor(0x7F, dtype=torch.uint8))
        return (codes if self.kv_layout == "hnd" else codes.transpose(1, 2)).contiguous().cuda()

    def slot(self, which, b, t, h):
        """A view of one token's codes of kv head h (8-bit formats)."""
        page = int(self.table[b, t // 16])
        pool = self.k if which == "k" else self.v
        return pool[page, h, t % 16] if self.kv_layout == "hnd" else pool[page, t % 16, h]

    def values(self, pool, scale):
        """[sum of ctx, hkv, 128] in 64 bits."""
        p = pool.cpu().numpy()
        if self.kv_dtype == "e2m1":
            p = np.asarray(e2m1.decode_slices(p), np.float64)
        else:
            p = attention.code_table(self.kv_dtype).astype(np.float64)[p]
            if self.kv_layout == "nhd":
                p = p.swapaxes(1, 2)
        rows = [p[self.table[b, :(c + 15) // 16]].swapaxes(1, 2).reshape(-1, self.hkv, 128)[:c]
                for b, c in enumerate(self.ctx)]
        return torch.from_numpy(np.concatenate(rows)).cuda() * float(np.float32(scale))

    @property
    def kind(self):
        return dict(kv_dtype=self.kv_dtype, kv_layout=self.kv_layout)


class Call:
    def __init__(self, new, ctx, hq=8, hkv=2, dtype="fp16", kv_dtype="e5m2", kv_layout="hnd", seed=0,
                 spread=1.0, pad=0, ks=1.0, vs=1.0, mbs=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.ctx, self.t, self.ks, self.vs = new, ctx, TYPES[dtype], ks, vs
        self.cache = Cache(ctx, hkv, kv_dtype, kv_layout, seed, mbs=mbs)
        self.q = (torch.randn(sum(new) + pad, hq, 128, device="cuda", generator=g) * spread).to(self.t)
        self.cu = offsets(new)
        self.lse = torch.full(self.q.shape[:2], 77.0, device="cuda")

    def run(self, causal=True, status=xqa.XQA_OK, **kw):
        c = self.cache
        self.shape = xqa.make_extend_shape(self.q, c.k, c.bt, causal=causal, **c.kind, **kw)
        self.ws = xqa.alloc_extend_workspace(self.shape)
        out = torch.full(self.q.shape, 55.0, dtype=self.t, device="cuda")
        xqa.xqa_extend(self.q, c.k, c.v, c.bt, c.lens, self.cu, self.ks, self.vs, out=out,
                       lse=self.lse, workspace=self.ws, shape=self.shape)
        torch.cuda.synchronize()
        assert xqa.xqa_read_status(self.ws) == status
        assert not bool(self.ws[64:64 + 8192].any())  # tickets back at zero
        return out

    def want(self, causal=True, sm_scale=None):
        c = self.cache
        return plain(self.q, c.values(c.k, self.ks), c.values(c.v, self.vs), self.new, self.ctx, causal,
                     sm_scale)

    def check(self, out, causal=True, sm_scale=None):
        n = sum(self.new)
        want, lse, big = self.want(causal, sm_scale)
        compare(out[:n], want[:n], big[:n], self.t)
        self.check_lse(lse[:n])
        assert bool((out[n:] == 55.0).all()) and bool((self.lse[n:] == 77.0).all())

    def check_lse(self, lse):
        got = self.lse[:lse.shape[0]].double()
        assert torch.equal(torch.isnan(got), torch.isnan(lse))
        assert torch.equal(torch.isinf(got), torch.isinf(lse))
        fin = torch.isfinite(lse)
        err = (got - lse).abs()[fin]
        assert bool((err <= 2.0**-18 * (1 + lse[fin].abs())).all()), float(err.max())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
def test_formats(kv_dtype, kv_layout, dtype):
    c = Call([5, 1, 40, 0, 130], [77, 300, 40, 19, 500], dtype=dtype, kv_dtype=kv_dtype,
             kv_layout=kv_layout, seed=3, pad=2, ks=0.5, vs=0.25)
    c.check(c.run())


@pytest.mark.parametrize("new,ctx", [([1], [1]), ([1], [16]), ([1], [17]), ([2], [2]), ([5], [705]),
                                     ([16], [128]), ([16], [129]), ([17], [127]), ([32], [256]),
                                     ([33], [2000]), ([128, 1], [128, 4096]), ([300, 5, 0, 64], [300, 5, 9, 64]),
                                     ([1000], [1000]), ([64], [1063])])
def test_lengths(new, ctx):
    c = Call(new, ctx, seed=len(new) + sum(ctx), pad=1)
    c.check(c.run())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (20, 4), (16, 1), (7, 1), (33, 1), (128, 1), (24, 3)])
def test_head_groups(hq, hkv, causal):
    c = Call([70, 1, 259], [170, 333, 259], hq=hq, hkv=hkv, seed=hq, dtype="bf16", kv_dtype="e4m3")
    c.check(c.run(causal), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx", [([50, 300], [20, 129]), ([40], [0]), ([3, 0, 9], [0, 0, 5]), ([256], [255])])
def test_fewer_tokens_than_queries(new, ctx, causal):
    # causal rows that see nothing are zero, their lse -inf
    c = Call(new, ctx, hq=12, hkv=4, seed=sum(ctx))
    c.check(c.run(causal), causal)


@pytest.mark.parametrize("max_ctas", [1, 2, 7, 0])
def test_shares_of_the_line(max_ctas):
    g = np.random.default_rng(5)
    new = [int(x) for x in g.integers(0, 60, 40)]
    ctx = [int(n + x) for n, x in zip(new, g.integers(0, 900, 40))]
    c = Call(new, ctx, hq=4, hkv=2, seed=9, kv_dtype="e4m3", kv_layout="nhd")
    c.check(c.run(max_ctas=max_ctas))


def test_more_sequences_than_threads():
    g = np.random.default_rng(6)
    new = [int(x) for x in g.integers(0, 4, 1500)]
    ctx = [int(n + x) for n, x in zip(new, g.integers(0, 40, 1500))]
    c = Call(new, ctx, hq=2, hkv=1, seed=10)
    c.check(c.run())


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
@pytest.mark.parametrize("new,ctx", [([1], [9000]), ([3, 2], [6001, 7000]), ([40, 1, 500], [5000, 9000, 3500])])
def test_pieces_of_long_contexts(new, ctx, kv_dtype, kv_layout):
    c = Call(new, ctx, kv_dtype=kv_dtype, kv_layout=kv_layout, seed=sum(new), dtype="bf16", vs=0.7129)
    c.check(c.run())


@pytest.mark.parametrize("max_ctas", [40, 1024])
def test_a_unit_in_tens_and_hundreds_of_pieces(max_ctas):
    c = Call([20], [140000], hq=8, hkv=1, seed=12, kv_dtype="e4m3")
    c.check(c.run(max_ctas=max_ctas))


def test_custom_scales_views_and_device_scales():
    c = Call([33, 70], [400, 70], hq=8, hkv=2, seed=21, ks=0.2937, vs=1.7)
    wide = torch.zeros(103, 12, 128, dtype=c.t, device="cuda")
    wide[:, :8] = c.q
    c.q = wide[:, :8]
    want = c.run(sm_scale=0.05)
    c.check(want, sm_scale=0.05)
    k = c.cache
    holder = torch.full((103, 10, 128), 3.0, dtype=c.t, device="cuda")
    out = holder[:, 1:9]
    xqa.xqa_extend(c.q, k.k, k.v, k.bt, k.lens, c.cu, torch.tensor([0.2937], device="cuda"),
                   torch.tensor([1.7], device="cuda"), out=out, sm_scale=0.05, **k.kind)
    assert torch.equal(out, want)
    assert bool((holder[:, 0] == 3.0).all()) and bool((holder[:, 9] == 3.0).all())


@pytest.mark.parametrize("spread", [30.0, 3000.0])
def test_large_logits_move_the_maximum(spread):
    c = Call([90, 3], [700, 1500], spread=spread, seed=4)
    out = c.run()
    # logits of up to 1e5 and more: 2^-23 of them is what the weights may be off by, relative
    want, _, big = c.want()
    u = torch.finfo(c.t).eps / 2
    reach = spread * 128 * 5 / math.sqrt(128) * 2.0**-23 * 8
    assert bool(((out[:93].double() - want).abs() <= (1.05 * u + reach) * (big[..., None] + want.abs()) + 1e-6).all())


@pytest.mark.parametrize("kv_dtype,bad", [("e5m2", 0x7C), ("e5m2", 0xFC), ("e5m2", 0x7F), ("e4m3", 0x7F)])
@pytest.mark.parametrize("at", [37, 127, 128, 199, 150])
def test_hidden_values_stay_hidden(kv_dtype, bad, at):
    """A value that is not finite reaches the rows that see its token, and no others."""
    c = Call([80, 40], [200, 300], kv_dtype=kv_dtype, seed=at)
    c.cache.slot("v", 0, at, 1)[5] = bad
    c.check(c.run())
    c.cache.slot("v", 0, at, 1)[5] = 0
    c.cache.slot("k", 0, at, 0)[7] = 0x7F  # a key of NaN
    out = c.run()
    seen = torch.zeros(120, dtype=torch.bool, device="cuda")
    seen[max(0, at - 120):80] = True
    got = torch.isnan(out).all(dim=-1)
    assert torch.equal(got[:, :4], seen[:, None].expand(120, 4)) and not bool(got[:, 4:].any())
    assert torch.equal(torch.isnan(c.lse), got)


def test_hidden_groups_of_a_4_bit_cache():
    c = Call([80], [200], kv_dtype="e2m1", seed=2)
    page = int(c.cache.table[0, 150 // 16])
    c.cache.v[page, 1, 1024 + (150 % 16) * 8 + 3] = 0x7F  # token 150, dims 48 .. 63
    out = c.run()
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[30:, 4:, 48:64] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
def test_pieces_with_hidden_and_visible_infinities(kv_dtype, kv_layout):
    c = Call([9, 2], [5000, 100], kv_dtype=kv_dtype, kv_layout=kv_layout, seed=8)
    good = c.run()
    pool = c.cache.v
    page, slot = int(c.cache.table[0, 4995 // 16]), 4995 % 16
    if kv_dtype == "e2m1":
        pool[page, 0, 1024 + slot * 8:1024 + slot * 8 + 8] = 0x7F
    elif kv_layout == "hnd":
        pool[page, 0, slot] = 0x7F
    else:
        pool[page, slot, 0] = 0x7F
    out = c.run()
    nan = torch.isnan(out)
    assert bool(nan[4:9, :4].all()) and int(nan.sum()) == 5 * 4 * 128
    assert torch.equal(out[:4], good[:4]) and torch.equal(out[9:], good[9:])


@pytest.mark.parametrize("bad", [-1, 10**6, 2**31 - 1, -(2**31)])
@pytest.mark.parametrize("at", [3, 15, 17])
def test_bad_pages(bad, at):
    """The rows that see a token of the page are NaN; the others are as without it."""
    c = Call([80, 20], [300, 100], seed=1)
    good = c.run()
    c.cache.bt[0, at] = bad
    out = c.run(status=xqa.XQA_ERR_BAD_BLOCK_ID)
    first = max(0, at * 16 - 220)
    assert bool(torch.isnan(out[first:80]).all()) and bool(torch.isnan(c.lse[first:80]).all())
    assert torch.equal(out[:first], good[:first]) and torch.equal(out[80:], good[80:])


@pytest.mark.parametrize("length", [-1, 321, 2**31 - 1])
def test_bad_lengths(length):
    c = Call([80, 20], [300, 100], seed=1, mbs=20)
    want, _, big = c.want()
    c.cache.lens[0] = length
    out = c.run(status=xqa.XQA_ERR_CTX_TOO_LONG)
    assert bool(torch.isnan(out[:80]).all()) and bool(torch.isnan(c.lse[:80]).all())
    compare(out[80:], want[80:], big[80:], c.t)


def test_bad_offsets_are_reported_and_contained():
    # (without a sequence the long ones are cut elsewhere: held against the definition)
    c = Call([10, 20, 30], [100, 200, 300], seed=1)
    want, _, big = c.want()
    for cu, good in (([0, 10, 30, 61], slice(0, 30)),    # past the rows
                     ([0, 60, 0, 60], slice(0, 0)),      # overlapping: more rows than there are
                     ([-5, 10, 30, 60], slice(10, 60)),
                     ([0, 10, 5, 35], slice(0, 5)),      # descending; the last one overlaps the first
                     ([0, 10, 30, 2**31 - 1], slice(0, 30))):
        c.cu = i32(cu)
        out = c.run(status=xqa.XQA_ERR_BAD_OFFSETS)
        compare(out[good], want[good], big[good], c.t)
        left = torch.ones(60, dtype=torch.bool, device="cuda")
        left[good] = False
        if cu != [0, 10, 5, 35]:
            assert bool((out[left] == 55).all())


@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, math.nan])
def test_a_device_scale_that_cannot_be(scale):
    c = Call([10, 20], [100, 200], seed=1)
    c.ks = torch.tensor([scale], device="cuda")
    out = c.run(status=xqa.XQA_ERR_VALUE)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(c.lse).all())


def test_graph_replay_with_other_lengths_and_streams():
    c = Call([8, 30, 2], [600, 2000, 50], seed=12, mbs=200, pad=20)
    k = c.cache
    shape = xqa.make_extend_shape(c.q, k.k, k.bt)
    ws = xqa.alloc_extend_workspace(shape)
    out = torch.zeros_like(c.q)
    call = lambda: xqa.xqa_extend(c.q, k.k, k.v, k.bt, k.lens, c.cu, 1.0, 1.0, out=out, lse=c.lse,
                                  workspace=ws, shape=shape)
    call()
    first = out.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # other lengths, in the same tensors
    c.new, c.ctx = [20, 3, 37], [555, 1500, 49]
    k.ctx = c.ctx
    k.lens.copy_(i32(c.ctx))
    c.cu.copy_(offsets(c.new))
    out.fill_(55.0)
    c.lse.fill_(77.0)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)
    assert xqa.xqa_read_status(ws) == xqa.XQA_OK


def test_two_calls_at_once_and_another_stream_without_a_workspace():
    a, b = Call([40, 3], [3000, 900], seed=1), Call([7], [5000], seed=2, kv_dtype="e4m3")
    want = [a.run(), b.run()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [xqa.xqa_extend(c.q, c.cache.k, c.cache.v, c.cache.bt, c.cache.lens, c.cu, 1.0, 1.0,
                               stream=s, **c.cache.kind) for c, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_one_workspace_for_every_attention_call():
    c = Call([4, 4], [700, 90], seed=5)
    k = c.cache
    shape = xqa.make_extend_shape(c.q, k.k, k.bt)
    q1 = c.q[[3, 7]].contiguous()
    ws = torch.zeros(max(xqa.xqa_extend_workspace_size(shape),
                         xqa.xqa_workspace_size(xqa.make_shape(q1, k.k, k.bt))),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out = xqa.xqa_extend(c.q, k.k, k.v, k.bt, k.lens, c.cu, 1.0, 1.0, workspace=ws, shape=shape)
        one = xqa.xqa_decode(q1, k.k, k.v, k.bt, k.lens, 1.0, 1.0, workspace=ws)
        want, _, big = c.want()
        compare(out, want, big, c.t)
        # decode's own tolerance: its weights are 32-bit sums of 16-bit products
        assert bool(((one.double() - want[[3, 7]]).abs() <= 2e-3 + 1e-2 * want[[3, 7]].abs()).all())


def test_binding_refusals():
    c = Call([10], [100], seed=1)
    k = c.cache
    args = lambda **kw: [kw.get("q", c.q), kw.get("k", k.k), kw.get("v", k.v), kw.get("bt", k.bt),
                         kw.get("lens", k.lens), kw.get("cu", c.cu), kw.get("ks", 1.0), kw.get("vs", 1.0)]
    for kw in (dict(q=c.q.float()), dict(q=c.q.cpu()), dict(q=c.q[:, :, :64]), dict(k=k.k.cpu()),
               dict(v=k.v[:2]), dict(bt=k.bt.long()), dict(lens=k.lens.long()), dict(cu=c.cu[:1]),
               dict(cu=c.cu.cpu()), dict(q=c.q.transpose(1, 2))):
        with pytest.raises((ValueError, xqa.XqaError)):
            xqa.xqa_extend(*args(**kw))
    for ks in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(xqa.XqaError) as e:
            xqa.xqa_extend(*args(ks=ks))
        assert e.value.code == xqa.XQA_ERR_VALUE
    shape = xqa.make_extend_shape(c.q, k.k, k.bt)
    with pytest.raises(ValueError):
        xqa.xqa_extend(*args(q=c.q[:5]), shape=shape)
    with pytest.raises(xqa.XqaError) as e:
        xqa.xqa_extend(*args(), shape=shape, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == xqa.XQA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        xqa.xqa_extend(*args(), lse=torch.zeros(3, 8, device="cuda"))
    empty = xqa.xqa_extend(c.q[:0], k.k, k.v, k.bt, k.lens, i32([0, 0]), 1.0, 1.0)
    assert empty.shape == (0, 8, 128)

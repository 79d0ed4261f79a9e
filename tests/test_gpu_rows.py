"""xqa_append and xqa_gather against the float64 formats of the oracle.

Codes are compared exactly: every quotient is formed in 32 bits and rounded to
the format, so a code can differ from the 64-bit definition only where the
quotient lies within 2^-22 of a rounding border (two 32-bit roundings, 2^-24
each, with room for a third). Scales that are powers of two and 16-bit inputs
meet no such border inexactly, and there every code must match.
"""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from oracle import e2m1, e4m3, e5m2

pytestmark = pytest.mark.gpu

FORMATS = [("e5m2", "hnd"), ("e5m2", "nhd"), ("e4m3", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")]
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
POISON = 0xA5


class Rows:
    """New rows of a few sequences and a poisoned cache for them."""

    def __init__(self, new, ctx, hkv, kv_dtype, kv_layout, dtype="fp16", seed=0, pad=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.ctx, self.hkv = new, ctx, hkv
        self.kv_dtype, self.kv_layout, self.t = kv_dtype, kv_layout, TYPES[dtype]
        pages = [(max(0, c) + 15) // 16 for c in ctx]
        self.nb, self.mbs = sum(pages) + 3, max(1, max(pages))
        order = rng.permutation(self.nb)
        self.table = np.full((len(ctx), self.mbs), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        n = sum(new) + pad
        mk = lambda: torch.from_numpy(rng.standard_normal((n, hkv, 128)) * np.exp(
            spread * rng.standard_normal((n, hkv, 1)))).cuda().to(self.t)
        self.k, self.v = mk(), mk()
        shape = {"e2m1": (self.nb, hkv, 1152)}.get(kv_dtype)
        shape = shape or ((self.nb, hkv, 16, 128) if kv_layout == "hnd" else (self.nb, 16, hkv, 128))
        self.kc = torch.full(shape, POISON, dtype=torch.uint8, device="cuda")
        self.vc = self.kc.clone()
        self.cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32).cuda()
        self.lens = torch.tensor(ctx, dtype=torch.int32).cuda()
        self.bt = torch.from_numpy(self.table).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, ks=1.0, vs=1.0, **kw):
        xqa.xqa_append(self.k, self.v, self.cu, self.kc, self.vc, self.bt, self.lens, ks, vs,
                       kv_dtype=self.kv_dtype, kv_layout=self.kv_layout, status=self.status, **kw)

    def gather(self, rows, ks=1.0, vs=1.0, cu=None, dtype=torch.float16, **kw):
        return xqa.xqa_gather(self.kc, self.vc, self.bt, self.lens, self.cu if cu is None else cu,
                              rows, ks, vs, dtype=dtype, kv_dtype=self.kv_dtype,
                              kv_layout=self.kv_layout, status=self.status, **kw)

    def places(self):
        """(row, page, slot) of every row that belongs in the cache."""
        row = 0
        for b, n in enumerate(self.new):
            for i in range(n):
                pos = self.ctx[b] - n + i
                yield row, int(self.table[b, pos // 16]), pos % 16
                row += 1

    def read(self, cache, page, slot):
        """The row's codes: uint8 [hkv, 128], or (codes, scales) in 4 bits."""
        c = cache[page]
        if self.kv_dtype == "e2m1":
            return c[:, 64 * slot:64 * slot + 64], c[:, 1024 + 8 * slot:1032 + 8 * slot]
        return c[:, slot] if self.kv_layout == "hnd" else c[slot]


def fp8_codes(x, scale, kv_dtype):
    """(codes, within 2^-22 of a border) by the 64-bit definition."""
    lut = (e5m2 if kv_dtype == "e5m2" else e4m3).lut()
    grid = lut[:124] if kv_dtype == "e5m2" else lut[:127]
    y = x / np.float64(np.float32(scale))
    mid = (grid[1:] + grid[:-1]) / 2
    j = np.searchsorted(mid, np.abs(y)).clip(0, len(mid) - 1)
    near = np.minimum(np.abs(np.abs(y) - mid[j]), np.abs(np.abs(y) - mid[np.maximum(j - 1, 0)]))
    code = e2m1.nearest_even(np.nan_to_num(np.abs(y), nan=0.0, posinf=np.inf), grid)
    return code + 128 * np.signbit(y), near <= np.abs(y) * 2.0**-22


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
@pytest.mark.parametrize("scales", [(1.0, 0.25), (0.2937, 0.7129)])
def test_append_writes_the_definitions_codes_and_nothing_else(kv_dtype, kv_layout, dtype, scales):
    r = Rows([1, 0, 37, 16, 3], [1, 5, 37, 49, 130], 3, kv_dtype, kv_layout, dtype, seed=3, pad=2)
    r.append(*scales)
    untouched = torch.ones_like(r.kc, dtype=torch.bool)
    exact = scales == (1.0, 0.25)
    for x, cache, scale in ((r.k, r.kc, scales[0]), (r.v, r.vc, scales[1])):
        x64, c = x.double().cpu().numpy(), cache.cpu().numpy()
        for row, page, slot in r.places():
            if kv_dtype == "e2m1":
                r.read(untouched, page, slot)[0].fill_(False)
                r.read(untouched, page, slot)[1].fill_(False)
                codes, sc = r.read(c, page, slot)
                wc, ws = e2m1.encode(x64[row], np.float64(np.float32(scale)))
                if exact:
                    assert np.array_equal(sc, ws) and np.array_equal(codes, wc), row
                else:  # a flipped border moves a value by one step of its group at most
                    a = e2m1.decode_slices(e2m1.pack(np.repeat(codes[:, None], 16, 1), np.repeat(sc[:, None], 16, 1)))
                    w = e2m1.decode_slices(e2m1.pack(np.repeat(wc[:, None], 16, 1), np.repeat(ws[:, None], 16, 1)))
                    assert np.mean(a != w) <= 1e-3
            else:
                r.read(untouched, page, slot).fill_(False)
                want, near = fp8_codes(x64[row], scale, kv_dtype)
                got = r.read(c, page, slot)
                diff = got != want
                assert not (diff & ~near).any(), (row, got[diff], want[diff])
                assert not exact or not diff.any()
    assert int(r.status.item()) == xqa.XQA_OK
    for cache in (r.kc, r.vc):
        assert bool((cache[untouched] == POISON).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv_dtype", ["e5m2", "e4m3"])
@pytest.mark.parametrize("scale", [1.0, 0.375, 0.2937, 2.0**-70, 1.7e9])
def test_every_16_bit_value_gets_the_code_of_the_32_bit_quotient(kv_dtype, dtype, scale):
    # all 65536 patterns; torch divides in 32 bits and rounds to the format
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).cuda().view(TYPES[dtype])
    r = Rows([128], [128], 4, kv_dtype, "nhd", dtype)
    r.k.copy_(bits.view(128, 4, 128))
    r.v.copy_(bits.flip(0).view(128, 4, 128))
    r.append(scale, scale)
    f8, big = (torch.float8_e5m2, 57344.0) if kv_dtype == "e5m2" else (torch.float8_e4m3fn, 448.0)
    pages = torch.from_numpy(r.table[0]).long().cuda()
    for x, cache in ((r.k, r.kc), (r.v, r.vc)):
        y = x.float() / torch.tensor(scale, dtype=torch.float32, device="cuda")
        want = y.clamp(-big, big).to(f8)
        got = cache[pages].view(128, 4, 128).view(f8)
        nan = torch.isnan(y)
        assert bool(torch.isnan(got.float())[nan].all())
        assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])


def test_4_bit_groups_of_special_values():
    r = Rows([16], [16], 1, "e2m1", "hnd")
    x = torch.randn(16, 1, 128, device="cuda").half()
    x[0, 0, 3] = float("nan")
    x[1, 0, 20] = float("inf")
    x[2, 0, 40] = -float("inf")
    x[3] = 0.0
    x[4, 0, :16] = 6e-8
    x[5, 0, :16] = 65504.0
    x[6, 0, 5] = -0.0
    r.k.copy_(x)
    r.append(1.0, 1.0)
    codes, scales = e2m1.encode(x.double().cpu().numpy()[:, 0], 1.0)
    page = r.kc.cpu().numpy()[int(r.table[0, 0]), 0]
    assert np.array_equal(page[1024:].reshape(16, 8), scales)
    keep = np.repeat(scales != 0x7F, 8, axis=1)  # codes of a NaN group stand for nothing
    assert np.array_equal(page[:1024].reshape(16, 64)[keep], codes[keep])
    back, _ = r.gather(16)
    assert bool(torch.isnan(back[0, 0, :16]).all()) and not bool(torch.isnan(back[0, 0, 16:]).any())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
def test_gather_reads_every_code(kv_dtype, kv_layout, dtype):
    # random bytes: every code of the format, NaN and infinities too; the value is formed in
    # 32 bits (one rounding of 2^-24) and rounded once: half a step of the type
    t = TYPES[dtype]
    r = Rows([33, 1, 0, 100], [33, 70, 9, 100], 2, kv_dtype, kv_layout, dtype, seed=5)
    rng = np.random.default_rng(7)
    r.kc.copy_(torch.from_numpy(rng.integers(0, 256, r.kc.shape, dtype=np.uint8)))
    r.vc.copy_(torch.from_numpy(rng.integers(0, 256, r.vc.shape, dtype=np.uint8)))
    ks, vs = 2.0**-6, 0.2937
    k, v = r.gather(134, ks, vs, dtype=t)
    for x, cache, scale in ((k, r.kc, ks), (v, r.vc, vs)):
        c, got = cache.cpu().numpy(), x.double().cpu().numpy()
        for row, page, slot in r.places():
            if kv_dtype == "e2m1":
                w = e2m1.decode_slices(c[page])[:, slot]
            else:
                w = (e5m2 if kv_dtype == "e5m2" else e4m3).lut()[r.read(c, page, slot)]
            w = w * np.float64(np.float32(scale))
            assert np.array_equal(np.isnan(got[row]), np.isnan(w))
            fin = np.isfinite(w) & (np.abs(w) < torch.finfo(t).max)
            assert np.array_equal(got[row][np.isinf(w)], w[np.isinf(w)])
            tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
            half = torch.finfo(t).eps / 2
            err = np.abs(got[row][fin] - w[fin])
            assert np.all(err <= np.abs(w[fin]) * (half + 2.0**-23) + tiny)
    assert int(r.status.item()) == xqa.XQA_OK


@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
def test_what_was_appended_is_gathered(kv_dtype, kv_layout):
    # append in two calls, gather whole: as if appended at once
    one = Rows([40, 7], [40, 7], 2, kv_dtype, kv_layout, "bf16", seed=9)
    one.append(0.5, 0.25)
    want = one.gather(47, 0.5, 0.25, dtype=torch.bfloat16)
    two = Rows([40, 7], [40, 7], 2, kv_dtype, kv_layout, "bf16", seed=9)
    full = (two.k, two.v)
    for cut, lens, rows in (([0, 33, 39], [33, 6], [*range(33), *range(40, 46)]),
                            ([0, 7, 8], [40, 7], [*range(33, 40), 46])):
        two.k, two.v = full[0][rows].contiguous(), full[1][rows].contiguous()
        two.cu = torch.tensor(cut, dtype=torch.int32).cuda()
        two.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        two.append(0.5, 0.25)
    got = two.gather(47, 0.5, 0.25, cu=one.cu, dtype=torch.bfloat16)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "nhd"), ("e2m1", "hnd")])
def test_views_with_strides(kv_dtype, kv_layout):
    r = Rows([5, 30], [9, 30], 4, kv_dtype, kv_layout, seed=11)
    want_k, want_v = r.kc.clone(), r.vc.clone()
    k, v = r.k.clone(), r.v.clone()
    r.append(0.5, 0.5)
    a, b = r.kc.clone(), r.vc.clone()
    qkv = torch.full((35, 12 + 8, 128), float("nan"), dtype=torch.float16, device="cuda")
    r.k, r.v = qkv[:, 12:16], qkv[:, 16:]
    r.k.copy_(k)
    r.v.copy_(v)
    r.kc.copy_(want_k)
    r.vc.copy_(want_v)
    r.append(0.5, 0.5)
    assert torch.equal(r.kc, a) and torch.equal(r.vc, b)
    # heads outermost, and written through a view
    r.k = k.transpose(0, 1).contiguous().transpose(0, 1)
    r.kc.copy_(want_k)
    r.append(0.5, 0.5)
    assert torch.equal(r.kc, a)
    plain = r.gather(35, 0.5, 0.5)
    wide = torch.full((40, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    r.gather(40, 0.5, 0.5, k=wide[:, :4], v=wide[:, 4:])
    assert torch.equal(wide[:35, :4], plain[0]) and torch.equal(wide[:35, 4:], plain[1])
    assert bool((wide[35:] == 7.0).all())  # rows behind the last sequence


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e4m3", "hnd"), ("e2m1", "hnd")])
def test_bad_lengths_and_pages_are_contained(kv_dtype, kv_layout):
    new, ctx = [4, 4, 4, 4, 20], [4, 4, 4, 4, 40]
    good = Rows(new, ctx, 2, kv_dtype, kv_layout, seed=13)
    good.append()
    want = good.gather(36)
    for kind in range(4):
        r = Rows(new, ctx, 2, kv_dtype, kv_layout, seed=13)
        lost = range(4 * kind, 4 * kind + 4) if kind < 3 else range(16 + 12, 16 + 20)
        if kind == 0:
            r.lens[0] = 3                    # fewer tokens than new ones
        elif kind == 1:
            r.lens[1] = -1
        elif kind == 2:
            r.lens[2] = 16 * r.mbs + 1
        else:                                # positions 32..39 of sequence 4
            r.bt[4, 2] = r.nb
        before = r.kc.clone()
        r.append()
        assert int(r.status.item()) == (xqa.XQA_ERR_BAD_BLOCK_ID if kind == 3 else xqa.XQA_ERR_CTX_TOO_LONG)
        keep = [i for i in range(36) if i not in lost]
        rows = list(good.places())
        for i in keep:
            _, page, slot = rows[i]
            a, b = r.read(r.kc, page, slot), r.read(good.kc, page, slot)
            assert all(torch.equal(x, y) for x, y in zip(a, b)) if kv_dtype == "e2m1" else torch.equal(a, b)
        for i in lost:
            _, page, slot = rows[i]
            a, b = r.read(r.kc, page, slot), r.read(before, page, slot)
            assert all(torch.equal(x, y) for x, y in zip(a, b)) if kv_dtype == "e2m1" else torch.equal(a, b)
        r.status.zero_()
        k, _ = r.gather(36)
        assert bool(torch.isnan(k[list(lost)]).all()) and torch.equal(k[keep], want[0][keep])
        assert int(r.status.item()) != xqa.XQA_OK


def test_offsets_that_do_not_ascend_touch_only_named_rows():
    r = Rows([8, 8, 8], [8, 8, 8], 1, "e5m2", "hnd")
    for cu in ([0, 20, 10, 24], [5, 5, 5, 5], [-7, -3, 8, 2000], [24, 16, 8, 0]):
        r.cu = torch.tensor(cu, dtype=torch.int32).cuda()
        r.append()
        r.gather(24)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kv_dtype", ["e4m3", "e2m1"])
def test_device_scales_graph_and_streams(kv_dtype):
    r = Rows([3, 30], [64, 30], 2, kv_dtype, "hnd", seed=15)
    r.append(0.5, 0.25)
    want = r.gather(33, 0.5, 0.25)
    ks, vs = torch.full((1,), 9.0, device="cuda"), torch.full((1,), 9.0, device="cuda")
    out = torch.zeros(33, 2, 128, dtype=torch.float16, device="cuda"), torch.zeros(33, 2, 128, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            r.append(ks, vs)
            r.gather(33, ks, vs, k=out[0], v=out[1])
    for a, b in ((0.5, 0.25), (0.3, 0.3), (0.5, 0.25)):
        ks.fill_(a)
        vs.fill_(b)
        r.kc.fill_(POISON)
        g.replay()
        torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    # a stream that is not the current one, ordered by the caller
    r.kc.fill_(POISON)
    side.wait_stream(torch.cuda.current_stream())
    r.append(0.5, 0.25, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    k, _ = r.gather(33, 0.5, 0.25)
    assert torch.equal(k, want[0])


def test_many_sequences_and_no_rows():
    rng = np.random.default_rng(17)
    new = rng.integers(0, 3, 700).tolist()
    ctx = [n + int(e) for n, e in zip(new, rng.integers(0, 40, 700))]
    r = Rows(new, ctx, 1, "e4m3", "hnd", seed=18)
    r.append()
    k, _ = r.gather(sum(new))
    ref = r.k.float().clamp(-448, 448).to(torch.float8_e4m3fn).to(torch.float16)
    assert torch.equal(k, ref)
    empty = Rows([0, 0], [3, 0], 1, "e5m2", "hnd")
    empty.append()
    assert empty.gather(0)[0].shape == (0, 1, 128)


def test_cache_past_4_gb():
    # page ids whose byte offsets pass 32 bits
    nb, hkv = 530_000, 4
    k = torch.randn(20, hkv, 128, device="cuda").half()
    table = torch.tensor([[nb - 1, nb - 7]], dtype=torch.int32).cuda()
    lens, cu = torch.tensor([20], dtype=torch.int32).cuda(), torch.tensor([0, 20], dtype=torch.int32).cuda()
    for kv_dtype, shape in (("e4m3", (nb, hkv, 16, 128)), ("e2m1", (nb * 2, hkv, 1152))):
        if kv_dtype == "e2m1":
            table = table + nb
        cache = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        assert cache.numel() > 2**32
        xqa.xqa_append(k, k, cu, cache, cache, table, lens, 1.0, 1.0, kv_dtype=kv_dtype)
        assert int(cache[: nb - 8].count_nonzero()) == 0
        a, _ = xqa.xqa_gather(cache, cache, table, lens, cu, 20, 1.0, 1.0, kv_dtype=kv_dtype)
        assert float((a - k).abs().max()) <= 0.17 * float(k.abs().max())
        del cache


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv_dtype,kv_layout", FORMATS)
@pytest.mark.parametrize("hkv", [4, 2, 5])
def test_many_rows_are_those_of_few(kv_dtype, kv_layout, dtype, hkv):
    # one call over many rows (two heads to a thread where they are even) writes the bytes
    # of calls over a sequence each, views with strides and bad entries among them
    new = [28000 // hkv, 8000 // hkv, 50]
    r = Rows(new, [new[0] + 77, new[1], 66], hkv, kv_dtype, kv_layout, dtype=dtype, seed=5, pad=3)
    r.bt[1, 3] = r.nb + 5
    wide = torch.zeros(r.k.shape[0], 3 * hkv, 128, dtype=r.k.dtype, device="cuda")
    wide[:, hkv:2 * hkv], wide[:, 2 * hkv:] = r.k, r.v
    k, v, cu, lens, bt = wide[:, hkv:2 * hkv], wide[:, 2 * hkv:], r.cu, r.lens, r.bt
    r.k, r.v = k, v
    r.append(0.3, 0.7)
    assert int(r.status[0]) == xqa.XQA_ERR_BAD_BLOCK_ID
    many = r.kc.clone(), r.vc.clone()
    r.kc.fill_(POISON)
    r.vc.fill_(POISON)
    at = 0
    for b, n in enumerate(new):
        r.k, r.v = k[at:at + n], v[at:at + n]
        r.cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        r.lens, r.bt = lens[b:b + 1].contiguous(), bt[b:b + 1].contiguous()
        r.append(0.3, 0.7)
        at += n
    assert torch.equal(r.kc, many[0]) and torch.equal(r.vc, many[1])

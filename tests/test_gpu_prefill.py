"""xqa_prefill against a plain float64 implementation.

Tolerances. Inputs are exact in both. Logits are 32-bit sums of 128 exact
products (relative error 2^-24 a step, far below what follows), weights 2^x and
their 32-bit sum are good to 2^-20. What remains:

* the weights are rounded to the type before the second product: half a step
  u = eps / 2 of each, so the row moves by at most u * sum_j w_j |v_j| <= u * max |v|
  over the keys it sees;
* the output is rounded once: u * |out|.

Together |got - out| <= 1.05 u (max |v| + |out|) + 1e-6, the factor and the last
term for the 32-bit parts. The log-sum-exp has no rounded weights: 2^-18 relative
to 1 + |lse|.
"""
import math

import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def offsets(lens):
    return torch.tensor([0, *np.cumsum(lens).tolist()], dtype=torch.int32).cuda()


def plain(q, k, v, lq, lk, causal, sm_scale=None):
    """(out, lse, bound's max |v|) in float64; hidden values never enter a sum."""
    hq, hkv = q.shape[1], k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    big = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    aq = ak = 0
    sm = sm_scale or 1 / math.sqrt(q.shape[2])
    for n, c in zip(lq, lk):
        if n and c:
            qs = q[aq:aq + n].double().transpose(0, 1).reshape(hkv, -1, q.shape[2])
            ks, vs = k[ak:ak + c].double().transpose(0, 1), v[ak:ak + c].double().transpose(0, 1)
            s = (qs @ ks.transpose(1, 2)).view(hq, n, c) * sm
            if causal:
                hidden = torch.ones(n, c, dtype=torch.bool, device="cuda").triu(c - n + 1)
                s = torch.where(hidden, torch.full_like(s, -math.inf), s)
            z = torch.logsumexp(s, dim=-1)
            w = torch.where(torch.isinf(z)[..., None] & (z[..., None] < 0), torch.zeros_like(s), torch.exp(s - z[..., None]))
            w = w.view(hkv, -1, c)
            clean = torch.where(torch.isfinite(vs), vs, torch.zeros_like(vs))
            o = w @ clean
            bad = ~torch.isfinite(vs)
            if bool(bad.any()):  # visible infinities and NaN reach the row, hidden ones do not
                seen = (w > 0).double()
                for val in (math.inf, -math.inf, math.nan):
                    is_val = torch.isnan(vs) if math.isnan(val) else vs == val
                    hit = (seen @ is_val.double()) > 0
                    o = torch.where(hit, o + val, o)
            rows = o.view(hq, n, -1)
            out[aq:aq + n] = rows.transpose(0, 1)
            lse[aq:aq + n] = z.transpose(0, 1)
            vmax = clean.abs().amax(dim=(1, 2)).repeat_interleave(hq // hkv)
            big[aq:aq + n] = vmax
        aq, ak = aq + n, ak + c
    return out, lse, big


class Call:
    def __init__(self, lq, lk=None, hq=8, hkv=2, dtype="fp16", seed=0, spread=1.0, pad=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        lk = lq if lk is None else lk
        self.lq, self.lk, self.t = lq, lk, TYPES[dtype]
        mk = lambda n, h: (torch.randn(n, h, 128, device="cuda", generator=g) * spread).to(self.t)
        self.q, self.k, self.v = mk(sum(lq) + pad, hq), mk(sum(lk) + pad, hkv), mk(sum(lk) + pad, hkv)
        self.cq, self.ck = offsets(lq), offsets(lk)
        self.lse = torch.full(self.q.shape[:2], 77.0, device="cuda")

    def run(self, causal=True, **kw):
        self.shape = xqa.make_prefill_shape(self.q, self.k, self.v, self.cq, causal=causal, **kw)
        self.ws = xqa.alloc_prefill_workspace(self.shape)
        out = torch.full(self.q.shape, 55.0, dtype=self.t, device="cuda")
        xqa.xqa_prefill(self.q, self.k, self.v, self.cq, self.ck, out=out, lse=self.lse,
                        workspace=self.ws, shape=self.shape)
        torch.cuda.synchronize()
        assert xqa.xqa_read_status(self.ws) == xqa.XQA_OK
        assert not bool(self.ws[:64].view(torch.int32)[4:].any())  # counters back at zero
        return out

    def check(self, out, causal=True, sm_scale=None):
        n = sum(self.lq)
        want, lse, big = plain(self.q[:n], self.k, self.v, self.lq, self.lk, causal, sm_scale)
        compare(out[:n], want, big, self.t)
        assert torch.equal(torch.isinf(self.lse[:n]), torch.isinf(lse.float()))
        fin = torch.isfinite(lse)
        err = (self.lse[:n].double() - lse).abs()[fin]
        assert bool((err <= 2.0**-18 * (1 + lse[fin].abs())).all()), float(err.max())
        assert bool((out[n:] == 55.0).all()) and bool((self.lse[n:] == 77.0).all())


def compare(out, want, big, t):
    u = torch.finfo(t).eps / 2
    got = out.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    fin = torch.isfinite(want)
    assert bool(torch.isfinite(got[fin]).all())
    bound = 1.05 * u * (big[..., None] + want.abs()) + 1e-6
    bad = ((got - want).abs() > bound) & fin
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first {i}: "
                             f"{float(got[i])} for {float(want[i])}, bound {float(bound[i])}")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2], [16], [37], [127, 1], [128], [129, 33], [300, 5, 0, 64], [1000]])
def test_whole_prompts(lens, dtype):
    c = Call(lens, dtype=dtype, seed=len(lens), pad=3)
    c.check(c.run())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (20, 4), (16, 1), (7, 1), (33, 1), (128, 1), (24, 3)])
def test_head_groups(hq, hkv, causal):
    c = Call([70, 1, 259], hq=hq, hkv=hkv, seed=hq, dtype="bf16")
    c.check(c.run(causal), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([1], [500]), ([3, 40], [130, 1027]), ([64, 10, 100], [64, 400, 0]),
                                   ([50, 300], [20, 129]), ([256, 256], [128, 255]), ([33], [4096])])
def test_other_numbers_of_keys_than_queries(lq, lk, causal):
    # more keys: a prompt that goes on; fewer: causal rows that see nothing are zero
    c = Call(lq, lk, hq=12, hkv=4, seed=sum(lk))
    c.check(c.run(causal), causal)


@pytest.mark.parametrize("max_ctas", [1, 3, 0])
def test_units_of_many_sequences(max_ctas):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 150).tolist()
    lens[40:75] = [0] * 35  # a whole chunk of the unit walk without a token
    c = Call(lens, hq=8, hkv=4, seed=5)
    c.check(c.run(max_ctas=max_ctas))


SPLIT = [([5], [3000]), ([1], [9001]), ([1, 30], [5000, 2]), ([16, 0, 40], [2500, 100, 4000]),
         ([3, 17], [4100, 900]), ([40], [5000])]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", SPLIT)
def test_few_queries_over_many_keys(lq, lk, causal, dtype):
    # units cut along the keys, pieces joined by the last CTA of a unit; among them
    # sequences with fewer tiles than pieces
    for hq, hkv in ((12, 4), (8, 1), (2, 2)):
        c = Call(lq, lk, hq=hq, hkv=hkv, seed=sum(lk), dtype=dtype, pad=2)
        out = c.run(causal)
        assert c.ws.numel() > 16384  # the pieces' place
        c.check(out, causal)
        assert not bool(c.ws[64:64 + 8 * 1024].any())  # the units' counts back at zero
        assert torch.equal(c.run(causal), out)


def test_pieces_with_hidden_and_visible_infinities():
    for at in (10, 2900, 2996, 2998):
        c = Call([5, 4], [3000, 1800], hq=8, hkv=2, seed=at)
        for val in (float("nan"), float("inf")):
            c.v[at, 1, 77] = val
            c.check(c.run())
        c = Call([5, 4], [3000, 1800], hq=8, hkv=2, seed=at)
        assert c.run() is not None and c.ws.numel() > 16384
        ref = c.run()
        c.k[at] = float("nan")
        out = c.run()
        assert c.ws.numel() > 16384
        first = max(0, at - 2995)
        assert bool(torch.isnan(out[first:5]).all())
        keep = [*range(first), *range(5, 9)]
        assert torch.equal(out[keep], ref[keep])
    c = Call([6], [2000], hq=4, hkv=2, seed=5)     # logits that move the maximum between pieces
    c.q.abs_()
    c.k.copy_(c.k[c.k[:, 0].float().sum(-1).argsort()] * 2)
    c.check(c.run())


def test_pieces_in_a_graph_with_other_lengths_and_bad_offsets():
    c = Call([9, 7], [3000, 2000], hq=8, hkv=2, seed=31)
    want = c.run()
    assert c.ws.numel() > 16384
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            xqa.xqa_prefill(c.q, c.k, c.v, c.cq, c.ck, out=out, workspace=c.ws, shape=c.shape)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    good_q, good_k = c.cq.clone(), c.ck.clone()
    c.cq.copy_(offsets([1, 15]))
    c.ck.copy_(offsets([4990, 10]))
    g.replay()
    torch.cuda.synchronize()
    w, _, big = plain(c.q, c.k, c.v, [1, 15], [4990, 10], True)
    compare(out, w, big, c.t)
    # bad key offsets: NaN rows; overlapping query offsets: reported, nothing out of place
    c.cq.copy_(good_q)
    c.ck.copy_(torch.tensor([0, 3000, 5001], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert xqa.xqa_read_status(c.ws) == xqa.XQA_ERR_BAD_OFFSETS
    assert torch.equal(out[:9], want[:9]) and bool(torch.isnan(out[9:]).all())
    for bad in ([0, 16, 0], [0, 16, 16], [3, 2, 1]):
        c.cq.copy_(torch.tensor(bad, dtype=torch.int32))
        g.replay()
    c.cq.copy_(good_q)
    c.ck.copy_(good_k)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and xqa.xqa_read_status(c.ws) == xqa.XQA_OK


def test_two_calls_in_pieces_at_once():
    a, b = Call([5], [40000], hq=8, hkv=2, seed=41), Call([8, 8], [9000, 12000], hq=8, hkv=2, seed=42)
    wa, wb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        oa, ob = torch.empty_like(wa), torch.empty_like(wb)
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
        xqa.xqa_prefill(a.q, a.k, a.v, a.cq, a.ck, out=oa, workspace=a.ws, shape=a.shape, stream=s1)
        xqa.xqa_prefill(b.q, b.k, b.v, b.cq, b.ck, out=ob, workspace=b.ws, shape=b.shape, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_one_long_prompt():
    c = Call([5000], hq=4, hkv=1, dtype="bf16", seed=6)
    c.check(c.run())


def test_large_logits_move_the_maximum():
    # logits up to +-100: the running maximum moves and O is rescaled; sorted keys make it
    # move in every tile
    for order in (1, -1):
        c = Call([700], hq=4, hkv=2, seed=7, spread=2.0)
        idx = c.k[:, 0, :].float().sum(-1).argsort()
        c.q.abs_()
        c.k.copy_(c.k[idx if order > 0 else idx.flip(0)])
        c.check(c.run())


def test_custom_scale_and_views_of_one_projection():
    c = Call([40, 90], hq=8, hkv=2, seed=8)
    want = c.run(sm_scale=0.02)
    c.check(want, sm_scale=0.02)
    qkv = torch.full((131, 12, 128), float("nan"), dtype=torch.float16, device="cuda")
    q, k, v = qkv[:130].split([8, 2, 2], dim=1)
    q.copy_(c.q), k.copy_(c.k), v.copy_(c.v)
    wide = torch.full((130, 10, 128), 3.0, dtype=torch.float16, device="cuda")
    got = xqa.xqa_prefill(q, k, v, c.cq, sm_scale=0.02, out=wide[:, 1:9])
    assert torch.equal(got, want)
    assert bool((wide[:, 0] == 3.0).all()) and bool((wide[:, 9] == 3.0).all())
    # heads outermost
    qt, kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k, c.v))
    assert torch.equal(xqa.xqa_prefill(qt, kt, vt, c.cq, sm_scale=0.02), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens,at", [([200, 150], 37), ([200, 150], 127), ([200, 150], 128), ([200, 150], 199),
                                     ([130, 400], 130 + 260), ([16, 16, 16], 20)])
def test_hidden_infinities_and_nan_stay_hidden(lens, at, dtype):
    # keys and values of one token that are not finite: rows that do not see it are as if it
    # were finite, rows that see it are not finite in those dims
    for hq, hkv in ((8, 2), (2, 2)):
        c = Call(lens, hq=hq, hkv=hkv, dtype=dtype, seed=at)
        for val in (float("nan"), float("inf"), float("-inf")):
            c.v[at, 0, 5] = val
            c.v[at, 1, 77] = val
            c.check(c.run())
        c.v[at, 0, 6] = float("inf")
        c.v[at, 0, 6 + 64] = float("nan")
        c.check(c.run())
        # a NaN key: rows that see it are NaN, others are untouched
        c = Call(lens, hq=hq, hkv=hkv, dtype=dtype, seed=at)
        ref = c.run()
        c.k[at] = float("nan")
        out = c.run()
        seq = int(np.searchsorted(np.cumsum(lens), at, side="right"))
        end = int(np.cumsum(lens)[seq])
        assert bool(torch.isnan(out[at:end]).all())
        keep = [i for i in range(sum(lens)) if not at <= i < end]
        assert torch.equal(out[keep], ref[keep])


def test_rows_behind_and_between_are_not_read():
    # NaN behind the last sequence, in q, k and v, changes nothing
    c = Call([100, 31], hq=8, hkv=2, seed=12, pad=9)
    want = c.run()
    c.check(want)
    for x in (c.q, c.k, c.v):
        x[131:] = float("nan")
    assert torch.equal(c.run(), want)
    # a gap between the key ranges of two sequences
    c = Call([60, 60], [90, 100], hq=8, hkv=2, seed=13)
    c.ck = torch.tensor([0, 90, 190], dtype=torch.int32).cuda()
    ref = c.run()
    c.k[60:90] = float("nan")
    c.v[60:90] = float("inf")
    c.lk = [60, 100]
    c.ck = torch.tensor([0, 60, 160], dtype=torch.int32).cuda()
    k, v = c.k, c.v
    c.k, c.v = torch.cat([k[:60], k[90:]]), torch.cat([v[:60], v[90:]])
    c.check(c.run())
    assert bool(torch.isfinite(ref).all())


def test_no_keys_and_no_rows():
    c = Call([5, 3], [0, 0])
    out = c.run()
    assert bool((out == 0).all()) and bool((c.lse == -math.inf).all())
    e = Call([0, 0])
    assert xqa.xqa_prefill(e.q, e.k, e.v, e.cq).shape == (0, 8, 128)


def test_bad_offsets_are_reported_and_contained():
    c = Call([40, 30, 20], hq=8, hkv=2, seed=14)
    want = c.run()
    good = c.cq.clone()
    for bad in ([0, 40, 70, 91], [0, 40, 30, 90], [-1, 40, 70, 90]):
        cq = torch.tensor(bad, dtype=torch.int32).cuda()
        out = torch.full_like(want, 9.0)
        xqa.xqa_prefill(c.q, c.k, c.v, cq, good, out=out, workspace=c.ws, shape=c.shape)
        assert xqa.xqa_read_status(c.ws) == xqa.XQA_ERR_BAD_OFFSETS
        lost = {91: slice(70, 90), 90: slice(40, 70) if bad[2] == 30 else slice(0, 40)}[bad[3]]
        keep = torch.ones(90, dtype=torch.bool, device="cuda")
        keep[lost] = False
        if bad[2] != 30:
            assert bool((out[~keep] == 9.0).all()) and torch.equal(out[keep], want[keep])
    for bad in ([0, 40, 70, 91], [0, 40, 39, 90], [-5, 40, 70, 90]):
        ck = torch.tensor(bad, dtype=torch.int32).cuda()
        out = xqa.xqa_prefill(c.q, c.k, c.v, good, ck, workspace=c.ws, shape=c.shape)
        assert xqa.xqa_read_status(c.ws) == xqa.XQA_ERR_BAD_OFFSETS
        seq = {91: 2, 90: 1 if bad[0] == 0 else 0}[bad[3]]
        lo, hi = [0, 40, 70][seq], [40, 70, 90][seq]
        assert bool(torch.isnan(out[lo:hi]).all())
        if seq != 1:
            keep = [i for i in range(90) if not lo <= i < hi]
            assert torch.equal(out[keep], want[keep])
    assert torch.equal(c.run(), want)


def test_graph_replay_streams_and_determinism():
    c = Call([120, 333], hq=8, hkv=2, seed=15)
    want = c.run()
    assert torch.equal(c.run(), want)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            for _ in range(3):
                xqa.xqa_prefill(c.q, c.k, c.v, c.cq, c.ck, out=out, workspace=c.ws, shape=c.shape)
    q = c.q.clone()
    for _ in range(2):
        c.q.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert not torch.equal(out, want)
        c.q.copy_(q)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    xqa.xqa_prefill(c.q, c.k, c.v, c.cq, c.ck, out=out, workspace=c.ws, shape=c.shape, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    # changed lengths at replay: offsets are read when the kernel runs
    c.cq.copy_(offsets([200, 253]))
    c.ck.copy_(offsets([200, 253]))
    g.replay()
    torch.cuda.synchronize()
    c.lq = c.lk = [200, 253]
    n, lse, big = plain(c.q, c.k, c.v, c.lq, c.lk, True)
    compare(out, n, big, c.t)


@pytest.mark.parametrize("dtype,q,k", [("bf16", 1e18, -1e16), ("bf16", 1e18, 1e16),
                                       ("fp16", 6e4, -6e4), ("fp16", 6e4, 6e4)])
def test_large_logits_are_a_softmax_like_any_other(dtype, q, k):
    # equal logits, near 1e36 with bf16 and 4e11 with fp16: means of the values
    c = Call([40], hq=2, hkv=1, dtype=dtype, seed=21)
    c.q.fill_(q)
    c.k.fill_(k)
    out = c.run()
    mean = c.v.double().cumsum(0) / torch.arange(1, 41, device="cuda").view(-1, 1, 1)
    u = torch.finfo(out.dtype).eps / 2
    assert float((out.double() - mean).abs().max()) <= 1.05 * u * 2 * float(c.v.abs().max()) + 1e-6


@pytest.mark.parametrize("hq,hkv", [(6, 2), (7, 1)])
def test_rows_do_not_depend_on_their_neighbours(hq, hkv):
    # a token with large logits beside others, whose rows come out as without it
    c = Call([60, 30], hq=hq, hkv=hkv, dtype="bf16", seed=25)
    want = c.run()
    c.q[20] *= 1e25
    got = c.run()
    assert torch.equal(got[:20], want[:20]) and torch.equal(got[21:], want[21:])
    assert bool(torch.isfinite(got[20]).all()) and not torch.equal(got[20], want[20])


@pytest.mark.parametrize("lk", [160, 1700])
def test_rows_past_32_bit_offsets(lk):
    # views whose rows lie 2^23 or 2^24 elements apart: the last ones past 2^31 elements,
    # in whole units and in units cut along the keys
    c = Call([150, 3], [lk, 20], hq=4, hkv=2, seed=26)
    want = c.run()
    n = max(153, lk + 20)
    big = torch.empty(n << 24 if lk < 1000 else n << 23, dtype=torch.float16, device="cuda").view(n, -1)
    q = big[:153, :512].view(153, 4, 128)
    out = big[:153, 512:1024].view(153, 4, 128)
    k = big[:lk + 20, 1024:1280].view(-1, 2, 128)
    v = big[:lk + 20, 1280:1536].view(-1, 2, 128)
    q.copy_(c.q), k.copy_(c.k), v.copy_(c.v)
    assert int(k.stride(0)) * (lk + 19) > 2**31
    xqa.xqa_prefill(q, k, v, c.cq, c.ck, out=out)
    assert torch.equal(out, want)


def test_another_stream_without_a_workspace():
    c = Call([70, 200], seed=22)
    want = c.run()
    side = torch.cuda.Stream()
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        got = xqa.xqa_prefill(c.q, c.k, c.v, c.cq, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)


def test_one_workspace_for_prompt_attention_and_decode():
    # alternately, also where units are cut into pieces; the counts and tickets stay zero
    a, b = Call([300], seed=23), Call([4], [5000], seed=24)
    wa, wb = a.run(), b.run()
    k = torch.randint(0, 60, (300, 2, 16, 128), dtype=torch.uint8, device="cuda")
    bt = torch.randperm(300, device="cuda").to(torch.int32).view(2, 150)
    lens = torch.tensor([2400, 900], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 8, 128, device="cuda").half()
    shape = xqa.make_shape(q, k, bt)
    ws = torch.zeros(max(xqa.xqa_workspace_size(shape), b.ws.numel()), dtype=torch.uint8, device="cuda")
    want = xqa.xqa_decode(q, k, k, bt, lens, 1.0, 1.0, workspace=ws, shape=shape).clone()
    for _ in range(3):
        for c, w in ((a, wa), (b, wb)):
            got = xqa.xqa_prefill(c.q, c.k, c.v, c.cq, c.ck, workspace=ws, shape=c.shape)
            assert torch.equal(got, w)
            assert torch.equal(xqa.xqa_decode(q, k, k, bt, lens, 1.0, 1.0, workspace=ws, shape=shape), want)


def test_two_calls_at_once_with_their_own_workspaces():
    a, b = Call([900], seed=16), Call([64, 700], seed=17)
    wa, wb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        oa = torch.empty_like(wa)
        ob = torch.empty_like(wb)
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
        xqa.xqa_prefill(a.q, a.k, a.v, a.cq, out=oa, workspace=a.ws, shape=a.shape, stream=s1)
        xqa.xqa_prefill(b.q, b.k, b.v, b.cq, out=ob, workspace=b.ws, shape=b.shape, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_binding_refusals():
    c = Call([8, 9])
    c.run()
    call = lambda **kw: xqa.xqa_prefill(**{**dict(q=c.q, k=c.k, v=c.v, cu_seqlens_q=c.cq), **kw})
    for kw, what in ((dict(q=c.q.float()), "dtype"), (dict(k=c.k.bfloat16()), "dtype"),
                     (dict(k=c.k[:, :1].expand(-1, 2, -1)), "stride"), (dict(v=c.v[1:]), "inconsistent"),
                     (dict(cu_seqlens_k=c.cq[:-1]), "batch"), (dict(lse=torch.zeros(3, 8, device="cuda")), "lse"),
                     (dict(out=torch.empty_like(c.q)[:, :4]), "match"),
                     (dict(shape=c.shape, q=c.q.transpose(0, 1).contiguous().transpose(0, 1)), "match"),
                     (dict(shape=c.shape, workspace=c.ws, k=c.k[1:], v=c.v[1:]), "match")):
        with pytest.raises(ValueError, match=what):
            call(**kw)
    with pytest.raises(xqa.XqaError):
        call(workspace=c.ws[:256])
    with pytest.raises(xqa.XqaError):
        x = torch.zeros(9, 3, 128, dtype=torch.float16, device="cuda")
        call(q=x[:8], k=x[:8, :2], v=x[:8, :2])

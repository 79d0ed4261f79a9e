"""The operators together, as a server uses them: prompts are attended to and their
keys and values written to the paged cache, a prompt goes on after its cached prefix,
and tokens are decoded one by one and two at a time over the same cache.

Every step is held against float64 attention over the values that the cache holds
(for the prompt: over the prompt's own keys and values), with the tolerances of the
operators' own tests.
"""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_prefill import compare, offsets, plain

pytestmark = pytest.mark.gpu

HQ, HKV = 8, 2


class Server:
    def __init__(self, lens, room, kv_dtype, kv_layout, seed):
        self.rng = torch.Generator(device="cuda").manual_seed(seed)
        self.kv_dtype, self.kv_layout = kv_dtype, kv_layout
        self.mbs = (max(lens) + room + 15) // 16
        self.nb = self.mbs * len(lens) + 3
        self.bt = torch.randperm(self.nb, device="cuda", generator=self.rng)[:self.mbs * len(lens)]
        self.bt = self.bt.to(torch.int32).view(len(lens), self.mbs).contiguous()
        shape = {"e2m1": (self.nb, HKV, 1152)}.get(kv_dtype)
        shape = shape or ((self.nb, HKV, 16, 128) if kv_layout == "hnd" else (self.nb, 16, HKV, 128))
        self.kc = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")  # NaN until written
        self.vc = self.kc.clone()
        self.lens = [0] * len(lens)
        self.ks, self.vs = 0.5, 0.25

    def rows(self, n, heads):
        return torch.randn(n, heads, 128, device="cuda", generator=self.rng).half()

    def context(self):
        return torch.tensor(self.lens, dtype=torch.int32).cuda()

    def append(self, k, v, new):
        self.lens = [a + b for a, b in zip(self.lens, new)]
        xqa.xqa_append(k, v, offsets(new), self.kc, self.vc, self.bt, self.context(), self.ks, self.vs,
                       kv_dtype=self.kv_dtype, kv_layout=self.kv_layout)

    def cached(self):
        return xqa.xqa_gather(self.kc, self.vc, self.bt, self.context(), offsets(self.lens),
                              sum(self.lens), self.ks, self.vs, kv_dtype=self.kv_dtype,
                              kv_layout=self.kv_layout)

    def decode(self, q):
        return xqa.xqa_decode(q, self.kc, self.vc, self.bt, self.context(), self.ks, self.vs,
                              kv_dtype=self.kv_dtype, kv_layout=self.kv_layout)


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
def test_prompts_continuations_and_tokens(kv_dtype, kv_layout):
    prompts = [37, 260, 5]
    s = Server(prompts, 80, kv_dtype, kv_layout, seed=len(kv_dtype))
    qkv = s.rows(sum(prompts), HQ + 2 * HKV)
    q, k, v = qkv.split([HQ, HKV, HKV], dim=1)
    out = xqa.xqa_prefill(q, k, v, offsets(prompts))
    s.append(k, v, prompts)
    want, _, big = plain(q, k, v, prompts, prompts, True)
    compare(out, want, big, torch.float16)
    # what the cache holds is near what was written: half a step of the format
    ck, cv = s.cached()
    step = {"e5m2": 2.0**-3, "e4m3": 2.0**-4, "e2m1": 2.0**-2}[kv_dtype]
    err = (cv.float() - v.float()).norm() / v.float().norm()
    assert float(err) <= step
    # the prompts go on: new rows attend to the cached prefix and themselves
    more = [20, 3, 41]
    qkv = s.rows(sum(more), HQ + 2 * HKV)
    q, k, v = qkv.split([HQ, HKV, HKV], dim=1)
    s.append(k, v, more)
    ck, cv = s.cached()
    out = xqa.xqa_prefill(q, ck, cv, offsets(more), offsets(s.lens))
    want, _, big = plain(q, ck, cv, more, s.lens, True)
    compare(out, want, big, torch.float16)
    # tokens, one and two at a time
    for n in (1, 1, 2, 1):
        new = [n] * 3
        s.append(s.rows(3 * n, HKV), s.rows(3 * n, HKV), new)
        q = s.rows(3 * n, HQ)
        got = s.decode(q if n == 1 else q.view(3, n, HQ, 128)).view(3 * n, HQ, 128)
        ck, cv = s.cached()
        want, _, big = plain(q, ck, cv, new, s.lens, True)
        # weights are summed as rounded: once more the output's share
        compare(got, want, big + want.abs().amax(-1), torch.float16)


def test_a_captured_step_of_append_and_decode():
    s = Server([64, 64], 40, "e2m1", "hnd", seed=3)
    s.append(s.rows(128, HKV), s.rows(128, HKV), [64, 64])
    k, v, q = s.rows(2, HKV), s.rows(2, HKV), s.rows(2, HQ)
    lens, cu = s.context(), offsets([1, 1])
    shape = xqa.make_shape(q, s.kc, s.bt, kv_dtype="e2m1")
    ws, out = xqa.alloc_workspace(shape), torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.add_(1)
        xqa.xqa_append(k, v, cu, s.kc, s.vc, s.bt, lens, s.ks, s.vs, kv_dtype="e2m1")
        xqa.xqa_decode(q, s.kc, s.vc, s.bt, lens, s.ks, s.vs, out=out, workspace=ws, shape=shape)
    for _ in range(20):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda", generator=s.rng))
        g.replay()
        torch.cuda.synchronize()
        s.lens = [n + 1 for n in s.lens]
        assert lens.tolist() == s.lens
        ck, cv = s.cached()
        want, _, big = plain(q, ck, cv, [1, 1], s.lens, True)
        compare(out, want, big + want.abs().amax(-1), torch.float16)


def test_gather_and_decode_on_another_stream():
    # outputs and workspaces that the binding allocates belong to the call's stream: the
    # zero fill of a workspace comes before the kernel that counts in it
    s = Server([900, 30], 20, "e4m3", "hnd", seed=8)
    s.append(s.rows(930, HKV), s.rows(930, HKV), [900, 30])
    q, cu, lens = s.rows(2, HQ), offsets(s.lens), s.context()
    want, (wk, wv) = s.decode(q), s.cached()
    side = torch.cuda.Stream()
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        got = xqa.xqa_decode(q, s.kc, s.vc, s.bt, lens, s.ks, s.vs, kv_dtype="e4m3", stream=side)
        k, v = xqa.xqa_gather(s.kc, s.vc, s.bt, lens, cu, 930, s.ks, s.vs, kv_dtype="e4m3", stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and torch.equal(k, wk) and torch.equal(v, wv)

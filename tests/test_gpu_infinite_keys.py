"""Keys whose logits are minus infinity (E5M2 and the 16-bit types have infinities): such a token has
weight 0, and a row that has no other is zero, its log-sum-exp minus infinity, in every attention
call. Held against float64 with the tolerances of each call's own tests; every query has a
positive value where the keys hold the infinity, so no logit is a NaN.
"""
import math

import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
import test_gpu_prefill as prompts
from gpu_helpers import ATOL, RTOL
from test_gpu_extend import Cache, Call
from test_gpu_prefill import plain

pytestmark = pytest.mark.gpu

DIM = 7
MINUS_INF = 0xFC  # E5M2


def positive(q):
    q[..., DIM] = q[..., DIM].abs() + 0.5


def hide(cache, b, first, last):
    """Minus infinity in the keys of a sequence's tokens first .. last - 1, of every head."""
    t = torch.arange(first, last, device="cuda")
    page = torch.from_numpy(cache.table[b]).cuda()[t // 16].long()
    if cache.kv_layout == "hnd":
        cache.k[page, :, t % 16, DIM] = MINUS_INF
    else:
        cache.k[page, t % 16, :, DIM] = MINUS_INF


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv_layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("new,ctx,hidden", [([80], [80], [30]),             # rows of one unit
                                            ([300, 9], [300, 700], [170, 700]),  # both row tiles; two chains
                                            ([20, 3], [9000, 200], [8990, 0]),   # pieces without a weight
                                            ([40, 5], [20, 0], [10, 0])])        # beside rows that see nothing
def test_chunks(new, ctx, hidden, dtype, kv_layout, causal):
    c = Call(new, ctx, hq=8, hkv=2, dtype=dtype, kv_layout=kv_layout, seed=sum(ctx), pad=1)
    positive(c.q)
    for b, n in enumerate(hidden):
        hide(c.cache, b, 0, n)
    out = c.run(causal)
    c.check(out, causal)
    if causal and new[0] <= ctx[0]:
        rows = hidden[0] - (ctx[0] - new[0])
        assert rows > 0 and bool((out[:rows] == 0).all()) and bool((c.lse[:rows] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lq,lk,hidden", [([80], [80], 30), ([300], [300], 170), ([64], [8256], 8210)])
def test_prompts(lq, lk, hidden, dtype):
    c = prompts.Call(lq, lk, hq=8, hkv=1, dtype=dtype, seed=hidden, pad=1)
    positive(c.q)
    c.k[:hidden, :, DIM] = -math.inf
    out = c.run()
    c.check(out)
    rows = hidden - (lk[0] - lq[0])
    assert rows > 0 and bool((out[:rows] == 0).all()) and bool((c.lse[:rows] == -math.inf).all())


@pytest.mark.parametrize("merge_mode", [0, 1])
@pytest.mark.parametrize("kv_layout", ["hnd", "nhd"])
@pytest.mark.parametrize("ctx,hidden", [([30, 5], [30, 0]), ([3000, 3000, 700], [3000, 2990, 690]), ([40000], [40000])])
def test_tokens(ctx, hidden, kv_layout, merge_mode):
    c = Cache(ctx, 2, "e5m2", kv_layout, seed=sum(ctx))
    for b, n in enumerate(hidden):
        hide(c, b, 0, n)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(len(ctx), 8, 128, device="cuda", generator=g).half()
    positive(q)
    shape = xqa.make_shape(q, c.k, c.bt, merge_mode=merge_mode, kv_layout=kv_layout)
    ws = xqa.alloc_workspace(shape)
    out = xqa.xqa_decode(q, c.k, c.v, c.bt, c.lens, 1.0, 1.0, workspace=ws, shape=shape)
    want, _, _ = plain(q, c.values(c.k, 1.0), c.values(c.v, 1.0), [1] * len(ctx), ctx, False)
    assert bool(((out.double() - want).abs() <= ATOL + RTOL * want.abs()).all())
    assert bool((out[0] == 0).all()) and xqa.xqa_read_status(ws) == xqa.XQA_OK

"""What xqa_extend leaves alone in a workspace: the merge tickets that decode and the choice of pages
keep there, zero between calls, are not its own."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
import test_gpu_prefill as prompts
from test_gpu_extend import Call
from test_gpu_prefill import compare

pytestmark = pytest.mark.gpu


def test_the_words_of_others_are_not_touched():
    c = Call([40, 3, 500], [5000, 9000, 3500], seed=4)  # units in pieces, units whole
    shape = xqa.make_extend_shape(c.q, c.cache.k, c.cache.bt)
    ws = xqa.alloc_extend_workspace(shape)
    words = ws[64:64 + 8192].view(torch.int32)
    words.copy_(torch.arange(1, 2049, device="cuda"))
    out = xqa.xqa_extend(c.q, c.cache.k, c.cache.v, c.cache.bt, c.cache.lens, c.cu, 1.0, 1.0, workspace=ws, shape=shape)
    want, _, big = c.want()
    compare(out, want, big, c.t)
    assert torch.equal(words, torch.arange(1, 2049, device="cuda", dtype=torch.int32))


def test_prompts_and_chunks_on_one_workspace_in_turn():
    c = Call([40, 3, 500], [5000, 9000, 3500], seed=4, dtype="bf16")
    p, cut = prompts.Call([300, 20, 700], dtype="bf16", seed=1), prompts.Call([64], [8256], hq=32, hkv=4, seed=2)
    eshape = xqa.make_extend_shape(c.q, c.cache.k, c.cache.bt)
    shapes = [xqa.make_prefill_shape(x.q, x.k, x.v, x.cq) for x in (p, cut)]
    ws = torch.zeros(max(xqa.xqa_extend_workspace_size(eshape), *map(xqa.xqa_prefill_workspace_size, shapes)),
                     dtype=torch.uint8, device="cuda")
    want, _, big = c.want()
    for _ in range(2):
        for x, shape in zip((p, cut), shapes):
            out = xqa.xqa_prefill(x.q, x.k, x.v, x.cq, x.ck, lse=x.lse, workspace=ws, shape=shape)
            x.check(out)
            assert xqa.xqa_read_status(ws) == xqa.XQA_OK
            out = xqa.xqa_extend(c.q, c.cache.k, c.cache.v, c.cache.bt, c.cache.lens, c.cu, 1.0, 1.0,
                                 workspace=ws, shape=eshape)
            compare(out, want, big, c.t)
            assert xqa.xqa_read_status(ws) == xqa.XQA_OK

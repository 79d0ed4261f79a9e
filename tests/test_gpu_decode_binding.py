"""The decode binding refuses, and launches nothing for, tensors that do not belong together."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv_dtype", ["e5m2", "e2m1"])
def test_refusals(kv_dtype):
    page = (2, 1152) if kv_dtype == "e2m1" else (2, 16, 128)
    q = torch.zeros(2, 8, 128, dtype=torch.float16, device="cuda")
    k = torch.zeros(6, *page, dtype=torch.uint8, device="cuda")
    bt = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    lens = torch.full((2,), 40, dtype=torch.int32, device="cuda")
    shape = xqa.make_shape(q, k, bt, kv_dtype=kv_dtype)
    ws, out = xqa.alloc_workspace(shape), torch.full_like(q, 3.0)
    good = dict(q=q, k_cache=k, v_cache=k.clone(), block_tables=bt, context_lens=lens, k_scale=1.0,
                v_scale=1.0, out=out, shape=shape)
    other = (2, 16, 128) if kv_dtype == "e2m1" else (2, 1152)
    bad = (dict(v_cache=k[:5]), dict(k_cache=k[:5]), dict(v_cache=torch.zeros(6, *other, dtype=torch.uint8, device="cuda")),
           dict(context_lens=lens[:1]), dict(block_tables=bt[:1]), dict(block_tables=bt[:, :2].contiguous()),
           dict(q=q[:1]), dict(out=out[:1]), dict(context_lens=lens.long()), dict(v_cache=k.cpu()),
           dict(q=q.transpose(0, 1)))
    for kw in bad:
        a = {**good, **kw}
        for call in (lambda: xqa.xqa_decode(**a, workspace=ws), lambda: xqa.xqa_attend_partial(**a, workspace=ws),
                     lambda: xqa.xqa_decode_static_workspace(**a)):
            with pytest.raises(ValueError):
                call()
        if "out" not in kw and "q" not in kw:  # without a descriptor: the tensors against one another
            with pytest.raises(ValueError):
                xqa.xqa_decode(**{**a, "shape": xqa.make_shape(q, k, bt, kv_dtype=kv_dtype)})
    with pytest.raises(ValueError):
        xqa.xqa_attend_partial(**good, workspace=None)
    for call in (lambda: xqa.xqa_plan(lens[:1], ws, shape), lambda: xqa.xqa_plan(None, ws, shape),
                 lambda: xqa.xqa_combine(lens, 1.0, out[:1], ws, shape),
                 lambda: xqa.xqa_combine(lens, 1.0, None, ws, shape)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    xqa.xqa_decode(**good, workspace=ws)
    xqa.xqa_decode(**{**good, "context_lens": torch.cat([lens, lens]), "block_tables": torch.cat([bt, bt])}, workspace=ws)
    torch.cuda.synchronize()
    assert bool((out == 0.0).all()) and xqa.xqa_read_status(ws) == xqa.XQA_OK


def test_any_object_with_a_stream_handle():
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    q = torch.randn(1, 8, 128, device="cuda").half()
    k = torch.randint(0, 100, (3, 2, 16, 128), dtype=torch.uint8, device="cuda")
    bt = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    shape = xqa.make_shape(q, k, bt)
    ws, out = xqa.alloc_workspace(shape), torch.zeros_like(q)
    want = xqa.xqa_decode(q, k, k, bt, lens, 1.0, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xqa.xqa_decode(q, k, k, bt, lens, 1.0, 1.0, out=out, workspace=ws, shape=shape, stream=Handle(side))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and xqa.xqa_read_status(ws, stream=Handle(side)) == xqa.XQA_OK

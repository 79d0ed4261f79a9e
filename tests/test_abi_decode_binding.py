"""Host checks of the decode binding: tensors that are not what the shape descriptor says are
refused before the library is called (no GPU: shapes alone, and CPU tensors)."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa

B, HQ, HKV, NB, MBS = 3, 8, 2, 20, 5
CACHES = {("e5m2", "hnd"): (NB, HKV, 16, 128), ("e4m3", "nhd"): (NB, 16, HKV, 128),
          ("e2m1", "hnd"): (NB, HKV, 1152)}


def fits(kv_dtype, kv_layout, q_len=1, **kw):
    page = CACHES[kv_dtype, kv_layout]
    shape = xqa.XqaShape(B, HQ, HKV, 128, 16, MBS, NB, 0.0, 0, 0, 0, xqa.KV_DTYPES[kv_dtype],
                         xqa.KV_LAYOUTS[kv_layout], q_len)
    q = (B, HQ, 128) if q_len == 1 else (B, q_len, HQ, 128)
    a = dict(q=q, k=page, v=page, bt=(B, MBS), lens=B, out=B * q_len * HQ * 128)
    a.update(kw)
    return xqa._decode_fits(bytes(shape), torch.Size(a["q"]), torch.Size(a["k"]), torch.Size(a["v"]),
                            torch.Size(a["bt"]), a["lens"], a["out"])


@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("kv_dtype,kv_layout", CACHES)
def test_tensors_that_fit(kv_dtype, kv_layout, q_len):
    page = CACHES[kv_dtype, kv_layout]
    assert fits(kv_dtype, kv_layout, q_len)
    # buffers with room for more pages and sequences than the call's
    assert fits(kv_dtype, kv_layout, q_len, k=(NB + 1, *page[1:]), v=(NB + 9, *page[1:]), bt=(B + 4, MBS), lens=B + 4)


@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("kv_dtype,kv_layout", CACHES)
def test_tensors_that_do_not_fit(kv_dtype, kv_layout, q_len):
    page = CACHES[kv_dtype, kv_layout]
    others = [c for c in CACHES.values() if c != page]
    for name in ("k", "v"):
        for c in (*others, (NB - 1, *page[1:]), (NB, HKV + 1, *page[2:]), (NB * HKV, *page[2:])):
            with pytest.raises(ValueError, match=name + "_cache"):
                fits(kv_dtype, kv_layout, q_len, **{name: c})
    for kw, what in ((dict(q=(B - 1, q_len, HQ, 128)), "q or out"), (dict(q=(B, q_len, HQ, 64)), "q or out"),
                     (dict(q=(B, q_len, 128, HQ)), "q or out"), (dict(out=B * q_len * HQ * 128 - 128), "q or out"),
                     (dict(bt=(B - 1, MBS)), "block_tables"), (dict(bt=(B, MBS - 1)), "block_tables"),
                     (dict(bt=(B, MBS + 1)), "block_tables"), (dict(bt=(B * MBS,)), "block_tables"),
                     (dict(lens=B - 1), "context_lens")):
        with pytest.raises(ValueError, match=what):
            fits(kv_dtype, kv_layout, q_len, **kw)


def test_cpu_tensors_are_refused_by_name():
    q = torch.zeros(B, HQ, 128, dtype=torch.float16)
    k = torch.zeros(CACHES["e5m2", "hnd"], dtype=torch.uint8)
    bt, lens = torch.zeros(B, MBS, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    shape = xqa.make_shape(q, k, bt)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        xqa.xqa_attend_partial(q, k, k, bt, lens, 1.0, 1.0, torch.empty_like(q), k, shape)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        xqa.xqa_decode_static_workspace(q, k, k, bt, lens, 1.0, 1.0)
    with pytest.raises(ValueError, match="context_lens"):
        xqa.xqa_plan(lens[:1], k, shape)
    with pytest.raises(ValueError, match="out"):
        xqa.xqa_combine(lens, 1.0, q[:1], k, shape)

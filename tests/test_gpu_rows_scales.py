"""xqa_append with scales that only the device knows, against quotients in 32 bits (each a
single IEEE division: equal bits)."""
import math

import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_rows import TYPES, Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv_dtype", ["e5m2", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.5, -0.2937, -(2.0**-70), 1e-40, math.inf, -math.inf, math.nan])
def test_device_scales_that_the_host_would_refuse(kv_dtype, dtype, scale):
    # the division as it is: all 65536 patterns of x
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).cuda().view(TYPES[dtype])
    r = Rows([128], [128], 4, kv_dtype, "nhd", dtype)
    r.k.copy_(bits.view(128, 4, 128))
    r.v.copy_(bits.flip(0).view(128, 4, 128))
    dev = torch.full((1,), scale, device="cuda")
    r.append(dev, dev)
    assert int(r.status.item()) == xqa.XQA_OK
    f8, big = (torch.float8_e5m2, 57344.0) if kv_dtype == "e5m2" else (torch.float8_e4m3fn, 448.0)
    pages = torch.from_numpy(r.table[0]).long().cuda()
    for x, cache in ((r.k, r.kc), (r.v, r.vc)):
        y = x.float() / dev
        want = y.clamp(-big, big).to(f8)
        got = cache[pages].view(128, 4, 128).view(f8)
        nan = torch.isnan(y)
        assert bool(torch.isnan(got.float())[nan].all())
        assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])


@pytest.mark.parametrize("kv_dtype,kv_layout", [("e5m2", "hnd"), ("e4m3", "nhd"), ("e2m1", "hnd")])
def test_a_negative_device_scale_reads_back(kv_dtype, kv_layout):
    # the format changes sign, what is read back does not
    r = Rows([40, 7], [40, 9], 2, kv_dtype, kv_layout, seed=3)
    r.append(0.3, 0.6)
    want = r.gather(47, 0.3, 0.6)
    ks, vs = torch.full((1,), -0.3, device="cuda"), torch.full((1,), -0.6, device="cuda")
    r.append(ks, vs)
    got = r.gather(47, ks, vs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool(got[0].any()) and bool(got[1].any())


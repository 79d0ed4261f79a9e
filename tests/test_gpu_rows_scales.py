"""xqa_append with scales that only the device knows, and the 4-bit codes of every group
maximum, against quotients in 32 bits (each a single IEEE division: equal bits)."""
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


def e2m1_code(y):
    """E2M1 codes (no sign) of the quotients |y|, to nearest even."""
    y = y.abs()
    return ((y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)).to(torch.uint8)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.375, 0.2937, 2.0**-70, 1.7e9])
def test_4_bit_codes_of_every_maximum_at_every_border(dtype, scale):
    # a group for each 16-bit magnitude (infinity too): its maximum, the values beside each
    # border of its codes and, in half of the groups, the signs turned
    t = TYPES[dtype]
    top = 0x7C00 if dtype == "fp16" else 0x7F80
    n = (top + 1 + 7) // 8 * 8
    mag = torch.arange(n, dtype=torch.int32, device="cuda").clamp(max=top)
    big = mag.to(torch.int16).view(t).float()
    one = torch.full((), scale, dtype=torch.float32, device="cuda")
    six = torch.full((), 6.0, device="cuda")  # (a number here would be multiplied by its reciprocal)
    s8 = (big / one / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    div = s * one
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    edge = torch.minimum(border * div[:, None], big[:, None])
    low = edge.to(t).view(torch.int16).int()
    low = low - (low.to(torch.int16).view(t).float() > edge).int()     # at or below the border
    pats = torch.cat([mag[:, None], low, torch.minimum(low + 1, mag[:, None]), 0 * mag[:, None]], 1)
    sign = (torch.arange(n * 16, device="cuda").view(n, 16) % 2 + torch.arange(n, device="cuda")[:, None] // 2) % 2
    x = (pats + sign.int() * 0x8000).to(torch.int16).view(t).view(n // 8, 1, 128)
    r = Rows([n // 8], [n // 8], 1, "e2m1", "hnd", dtype)
    r.k.copy_(x)
    r.v.copy_(x.flip(0))
    r.append(scale, scale)
    y = x.view(n, 16).float() / div[:, None]
    code = torch.where(s[:, None] > 0, e2m1_code(y), torch.zeros_like(y, dtype=torch.uint8)) + 8 * sign.to(torch.uint8)
    want = (code[:, 0::2] + 16 * code[:, 1::2]).view(n // 8, 64)
    pages = torch.from_numpy(r.table[0]).long().cuda()
    for cache, turn in ((r.kc, False), (r.vc, True)):
        c = cache[pages][:, 0]
        codes = c[:, :1024].reshape(-1, 64)[:n // 8]
        scales = c[:, 1024:].reshape(-1, 8)[:n // 8]
        w, ws = (want.flip(0), s8.view(torch.uint8).view(-1, 8).flip(0)) if turn else (want, s8.view(torch.uint8).view(-1, 8))
        assert torch.equal(scales, ws)
        bad = (codes != w).nonzero()
        assert len(bad) == 0, (len(bad), bad[0].tolist())

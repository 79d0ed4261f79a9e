"""xqa_select over tables that are too long for shared memory, and choices of more pages than its list
holds there, on bounds of random bytes. Choices are whole numbers: they have to equal a plain
implementation in 64 bits, however the work is split."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_extend import i32
from test_gpu_select import plain_select

pytestmark = pytest.mark.gpu

HKV, HQ = 2, 8


def random_bounds(g, nb):
    """[nb, HKV, 272]: lower below upper, exponents of a wide range, some slices without bounds."""
    b = np.sort(g.integers(-127, 128, (2, nb, HKV, 128)), axis=0).astype(np.int8)
    out = np.zeros((nb, HKV, 272), np.int8)
    out[..., :128], out[..., 128:256] = b[1], b[0]
    out[..., 256] = g.integers(-6, 3, (nb, HKV))
    odd = g.random((nb, HKV)) < 0.001
    out[odd] = 0
    out[odd, 256] = -128
    return torch.from_numpy(out.view(np.uint8)).cuda()


@pytest.mark.parametrize("max_ctas", [1, 0])
@pytest.mark.parametrize("nb", [997, None])  # every page many times (ties), or once
@pytest.mark.parametrize("pages", [8192, 8193, 20000, 70000])
def test_long_tables_and_many_pages(pages, nb, max_ctas):
    g = np.random.default_rng(pages + (nb or 0))
    nb = nb or pages
    bounds = random_bounds(g, nb)
    table = np.stack([np.concatenate([g.permutation(nb) for _ in range(-(-pages // nb))])[:pages] for _ in range(2)])
    table = table.astype(np.int32)
    ctx = [16 * pages - 3, 16 * (pages // 3) + 5]
    q = torch.from_numpy(g.standard_normal((2, HQ, 128))).half().cuda()
    bt, lens = torch.from_numpy(table).cuda(), i32(ctx)
    for k, first, last in ((100, 1, 2), (2048, 0, 1), (2049, 4, 16), (5000, 1, 1)):
        shape = xqa.make_select_shape(q, bounds, bt, k, first, last, max_ctas)
        ws = xqa.alloc_select_workspace(shape)
        want, wlens = plain_select(q, bounds, table, ctx, HKV, k, first, last)
        for _ in range(2):
            sel, sel_lens = xqa.xqa_select(q, bounds, bt, lens, workspace=ws, shape=shape)
            assert np.array_equal(sel_lens.cpu().numpy(), wlens)
            assert np.array_equal(sel.cpu().numpy(), want)
        assert xqa.xqa_read_status(ws) == xqa.XQA_OK


def test_scores_that_are_nearly_alike():
    """Keys that differ in their last bits alone, and a few that are far off: every round of the
    search for the last score narrows the range again."""
    pages = 12000
    g = np.random.default_rng(5)
    b = np.zeros((pages, HKV, 272), np.int8)
    b[..., 0] = 127
    b[..., 1] = g.integers(0, 3, (pages, HKV))
    b[::4000, :, 256] = 20
    b[1::4000, :, 256] = -20
    bounds = torch.from_numpy(b.view(np.uint8)).cuda()
    table = g.permutation(pages).astype(np.int32).reshape(1, -1)
    q = torch.zeros((1, HQ, 128), dtype=torch.float16, device="cuda")
    q[..., 0], q[..., 1] = 1.0, 1.0 / 64
    for k in (5, 700, 3000, 11999):
        sel, lens = xqa.xqa_select(q, bounds, torch.from_numpy(table).cuda(), i32([16 * pages]), k, 1, 1)
        want, wlens = plain_select(q, bounds, table, [16 * pages], HKV, k, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(lens.cpu().numpy(), wlens)

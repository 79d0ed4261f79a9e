"""The calls over pages with clusters of other sizes than the device's: a context that has no place
for 16 CTAs takes fewer. The library chooses by itself, so the unit is compiled here once more
with a way in."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from paged_fp8_kv_gqa_gb300 import build
from test_gpu_pages import Pool, i32, plain_assign, plain_release

pytestmark = pytest.mark.gpu

SHIM = r"""
#include "pages.cu"
extern "C" int shim_choice(int places) { return xqa::largest_cluster([&](int c) { return c <= places; }); }
extern "C" int shim_device() { int c = 0; return xqa::set_pages_attributes(&c) == cudaSuccess ? c : -1; }
extern "C" int shim_assign(void** a, int batch, int mbs, int nb, int rows, int cluster) {
  xqa::PagesParams p{};
  p.new_tokens = (const int32_t*)a[0], p.context_lens = (const int32_t*)a[1], p.block_tables = (int32_t*)a[2];
  p.free_pages = (int32_t*)a[3], p.num_free = (const int32_t*)a[4], p.new_lens = (int32_t*)a[5];
  p.new_free = (int32_t*)a[6], p.cu_seqlens = (int32_t*)a[7], p.slots = (int32_t*)a[8];
  p.positions = (int32_t*)a[9], p.status = (int32_t*)a[10];
  p.batch = batch, p.max_blocks_per_seq = mbs, p.num_blocks = nb, p.num_rows = rows;
  return (int)xqa::launch_assign(p, cluster, nullptr);
}
extern "C" int shim_release(void** a, int batch, int mbs, int nb, int cluster) {
  xqa::PagesParams p{};
  p.done = (const uint8_t*)a[0], p.context_lens = (const int32_t*)a[1], p.block_tables = (int32_t*)a[2];
  p.free_pages = (int32_t*)a[3], p.num_free = (const int32_t*)a[4], p.new_lens = (int32_t*)a[5];
  p.new_free = (int32_t*)a[6], p.status = (int32_t*)a[7];
  p.batch = batch, p.max_blocks_per_seq = mbs, p.num_blocks = nb;
  return (int)xqa::launch_release(p, cluster, nullptr);
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("shim")
    (d / "shim.cu").write_text(SHIM)
    subprocess.run([build.nvcc_path(), *build.ARCH_FLAGS, *build.NVCC_FLAGS, "-shared", "-cudart", "static",
                    str(d / "shim.cu"), "-o", str(d / "shim.so")], check=True, capture_output=True)
    torch.cuda.synchronize()
    so = ctypes.CDLL(str(d / "shim.so"))
    for name, ints in (("shim_assign", 5), ("shim_release", 4)):
        getattr(so, name).argtypes = [ctypes.POINTER(ctypes.c_void_p)] + [ctypes.c_int] * ints
    assert so.shim_device() in (1, 2, 4, 8, 16)
    return so


def pointers(*tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def test_the_largest_cluster_that_fits(shim):
    assert [shim.shim_choice(n) for n in (0, 1, 2, 7, 8, 15, 16, 40)] == [1, 1, 2, 4, 8, 8, 16, 16]


@pytest.mark.parametrize("cluster", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("batch,reach", [(65, 3000), (1500, 40)])
def test_every_size_gives_the_same(shim, cluster, batch, reach):
    if cluster > shim.shim_device():
        pytest.skip("the device has no place for such a cluster")
    g = np.random.default_rng(batch)
    ctx, new = ([int(x) for x in g.integers(0, n, batch)] for n in (reach, 90))
    done = [int(x) for x in g.integers(0, 2, batch)]
    mbs = (reach + 90 + 15) // 16
    pool = Pool(ctx, mbs, sum((c + n + 15) // 16 for c, n in zip(ctx, new)) + 9, seed=batch)
    rows = max(4097, sum(new)) + 3
    d, status, cu = pool.dev(), i32([0]), i32([0] * (batch + 1))
    slots, positions = i32([0] * rows), i32([0] * rows)
    lens, num, more = torch.zeros_like(d["lens"]), i32([0]), i32(new)
    torch.cuda.synchronize()
    assert shim.shim_assign(pointers(more, d["lens"], d["table"], d["free"], d["num"], lens, num, cu, slots,
                                     positions, status), batch, mbs, pool.nb, rows, cluster) == 0
    torch.cuda.synchronize()
    wlens, table, left, wcu, wslots, wpos, errors = plain_assign(pool, new, rows)
    assert not errors and int(status) == xqa.XQA_OK
    assert (lens.tolist(), num.tolist(), cu.tolist()) == (wlens, [left], wcu)
    assert np.array_equal(d["table"].cpu().numpy(), table)
    assert slots.tolist() == wslots and positions.tolist() == wpos
    d = pool.dev()
    flags = torch.tensor(done, dtype=torch.uint8).cuda()
    torch.cuda.synchronize()
    assert shim.shim_release(pointers(flags, d["lens"], d["table"], d["free"], d["num"], lens, num, status),
                             batch, mbs, pool.nb, cluster) == 0
    torch.cuda.synchronize()
    wlens, free, left, errors = plain_release(pool, done)
    assert not errors and int(status) == xqa.XQA_OK
    assert (lens.tolist(), num.tolist()) == (wlens, [left])
    assert np.array_equal(d["free"].cpu().numpy(), free)

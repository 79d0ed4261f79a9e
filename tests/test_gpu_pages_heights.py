"""xqa_release_pages where the free pages' number cannot be one: the call is refused whole, so no
page is lost and no free one overwritten."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_pages import Pool, i32, plain_release

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ctx,mbs", [([40, 33, 0, 7], 9), ([900, 33, 0, 7] * 300, 60)])  # one CTA, a cluster
@pytest.mark.parametrize("height", [-1, 1, 2**31 - 1, -(2**31)])
def test_a_height_that_cannot_be_releases_nothing(height, ctx, mbs, in_place):
    used = sum((c + 15) // 16 for c in ctx)
    pool = Pool(ctx, mbs, used + 20, seed=mbs)
    done = [b % 3 != 1 for b in range(len(ctx))]
    d, status = pool.dev(), i32([0])
    if height > 0:
        height = max(height, pool.nb + 1)
    d["num"].fill_(height)
    free = d["free"].clone()
    out = {} if in_place else dict(new_lens=torch.full_like(d["lens"], 7), new_free=i32([7]))
    call = lambda: xqa.xqa_release_pages(torch.tensor(done).cuda(), d["lens"], d["table"], d["free"], d["num"],
                                         status=status, **out)
    call()
    assert int(status) == xqa.XQA_ERR_NO_PAGES
    assert out.get("new_lens", d["lens"]).tolist() == ctx and out.get("new_free", d["num"]).tolist() == [height]
    assert torch.equal(d["free"], free)
    # the number put right, the same call gives every page back
    d["num"].fill_(pool.num_free)
    status.zero_()
    call()
    lens, want, left, _ = plain_release(pool, done)
    assert int(status) == xqa.XQA_OK and out.get("new_lens", d["lens"]).tolist() == lens
    assert out.get("new_free", d["num"]).tolist() == [left] and d["free"].tolist() == want.tolist()

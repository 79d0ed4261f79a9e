"""xqa_release_pages over the longest tables it takes: nearly 2^31 entries go through one list, the
last of them as well as the first."""
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa
from test_gpu_extend import i32

pytestmark = pytest.mark.gpu


def test_the_last_entries_of_the_longest_list():
    batch, mbs, nb = 16, 2**27 - 1, 3000
    table = torch.full((batch, mbs), -1, dtype=torch.int32, device="cuda")  # 8.6 GB of pages that are none
    order = torch.randperm(nb, device="cuda").to(torch.int32)
    table[0, 5:505] = order[:500]
    table[7, 2**26:2**26 + 400] = order[500:900]
    table[15, mbs - 1100:] = order[900:2000]
    lens, num = i32([16 * mbs] * batch), i32([0])
    free = torch.full((nb,), -5, dtype=torch.int32, device="cuda")
    xqa.xqa_release_pages(torch.ones(batch, dtype=torch.bool, device="cuda"), lens, table, free, num)
    assert int(num) == 2000 and torch.equal(free[:2000], order[:2000])
    assert bool((free[2000:] == -5).all()) and lens.tolist() == [0] * batch

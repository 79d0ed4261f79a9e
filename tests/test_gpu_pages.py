"""xqa_assign_pages and xqa_release_pages against one request after another in Python. All
results are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gqa_gb300 as xqa

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Pool:
    def __init__(self, ctx, mbs, nb, spare=None, seed=0):
        g = np.random.default_rng(seed)
        self.nb, self.mbs = nb, mbs
        ids = g.permutation(nb).astype(np.int32)
        self.table = np.full((len(ctx), mbs), -9, np.int32)
        at = 0
        for b, c in enumerate(ctx):
            p = min((max(c, 0) + 15) // 16, mbs)
            self.table[b, :p] = ids[at:at + p]
            at += p
        left = ids[at:] if spare is None else ids[at:at + spare]
        self.free = np.full(nb, -5, np.int32)
        self.free[:len(left)] = left
        self.num_free = len(left)
        self.ctx = list(ctx)

    def dev(self):
        return dict(lens=i32(self.ctx), table=torch.from_numpy(self.table).cuda(),
                    free=torch.from_numpy(self.free).cuda(), num=i32([self.num_free]))


def plain_assign(pool, new, rows):
    """(lens, table, num_free, cu, slots, positions, codes of the errors)"""
    table, lens, left = pool.table.copy(), list(pool.ctx), pool.num_free
    cu, slots, positions, errors = [0], [], [], set()
    asked_rows = asked_pages = 0
    for b, n in enumerate(new):
        c = lens[b]
        if n < 0 or c < 0 or c + n > pool.mbs * 16:
            errors.add(xqa.XQA_ERR_CTX_TOO_LONG)
            n = 0
        asked_rows += n
        if n and asked_rows > rows:
            errors.add(xqa.XQA_ERR_BAD_OFFSETS)
            n = 0
        need = (c + n + 15) // 16 - (c + 15) // 16 if n else 0
        asked_pages += need
        if need and asked_pages > pool.num_free:
            errors.add(xqa.XQA_ERR_NO_PAGES)
            n = 0
        for pos in range(c, c + n):
            if pos % 16 == 0:
                left -= 1
                table[b, pos // 16] = pool.free[left]
            slots.append(int(table[b, pos // 16]) * 16 + pos % 16)
            positions.append(pos)
        cu.append(cu[-1] + n)
        lens[b] = c + n
    pad = [-1] * (rows - len(slots))
    return lens, table, left, cu, slots + pad, positions + pad, errors


def check_assign(pool, new, rows, in_place=False):
    d = pool.dev()
    status = i32([0])
    out = dict(new_lens=torch.full_like(d["lens"], 7), new_free=i32([7])) if not in_place else {}
    cu, slots, positions = xqa.xqa_assign_pages(i32(new), d["lens"], d["table"], d["free"], d["num"],
                                                rows, status=status, **out)
    lens, table, left, wcu, wslots, wpos, errors = plain_assign(pool, new, rows)
    got = (out.get("new_lens", d["lens"]).tolist(), out.get("new_free", d["num"]).tolist(), cu.tolist())
    assert got == (lens, [left], wcu)
    assert np.array_equal(d["table"].cpu().numpy(), table)
    assert slots.tolist() == wslots and positions.tolist() == wpos
    assert np.array_equal(d["free"].cpu().numpy(), pool.free)
    if not in_place:
        assert d["lens"].tolist() == pool.ctx and d["num"].tolist() == [pool.num_free]
    code = int(status)
    assert code in errors if errors else code == xqa.XQA_OK


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ctx,new", [([0], [1]), ([16], [1]), ([15], [1]), ([15], [2]), ([0], [0]), ([31], [0]),
                                     ([0, 5, 16, 17], [16, 11, 16, 100]), ([3] * 9, [0, 1, 0, 13, 14, 0, 0, 40, 0]),
                                     ([100], [1000])])
def test_small_steps(ctx, new, in_place):
    pool = Pool(ctx, 80, 200, seed=len(ctx))
    check_assign(pool, new, sum(new), in_place)
    check_assign(pool, new, sum(new) + 5, in_place)


@pytest.mark.parametrize("batch,most,reach", [(7, 3, 100), (511, 1, 300), (512, 40, 200), (513, 200, 400),
                                              (1300, 30, 60), (3, 20000, 5)])
def test_many_sequences_and_rows(batch, most, reach):
    g = np.random.default_rng(batch)
    ctx = [int(x) for x in g.integers(0, reach, batch)]
    new = [int(x) for x in g.integers(0, most + 1, batch)]
    mbs = (max(ctx) + most + 15) // 16 + 1
    pool = Pool(ctx, mbs, sum((c + n + 15) // 16 for c, n in zip(ctx, new)) + 9, seed=batch)
    check_assign(pool, new, sum(new) + 3, in_place=bool(batch % 2))


def test_refusals_leave_the_others_served():
    pool = Pool([10, 70, 16, 0, 31, 5], 5, 40, spare=3)
    check_assign(pool, [1, 11, 16, 33, 1, 6], 100)      # 81 tokens are too many; 33 need 3 pages, 2 are left
    check_assign(pool, [-1, 10, 16, 16, 2, 6], 100, in_place=True)
    check_assign(pool, [6, 10, 16, 0, 1, 0], 20)        # rows run out at the third
    check_assign(pool, [6, 10, 16, 16, 1, 6], 100)      # pages run out; those that need none are served
    pool.ctx[0] = -4
    check_assign(pool, [6, 1, 1, 1, 1, 1], 100)
    many = Pool([0] * 1100, 4, 2000, spare=600)
    check_assign(many, [1] * 1100, 1100)
    check_assign(many, [1] * 1100, 550)


@pytest.mark.parametrize("height", [-1, 41, 2**31 - 1])
def test_a_height_that_cannot_be(height):
    pool = Pool([10, 16], 5, 40)
    d, status = pool.dev(), i32([0])
    d["num"].fill_(height)
    cu, slots, _ = xqa.xqa_assign_pages(i32([2, 2]), d["lens"], d["table"], d["free"], d["num"], 4,
                                        status=status)
    assert cu.tolist() == [0, 2, 2] and int(status) == xqa.XQA_ERR_NO_PAGES
    assert int(d["num"]) == 0 and d["lens"].tolist() == [12, 16]


def test_pages_that_are_none():
    pool = Pool([10, 16], 5, 40)
    pool.free[pool.num_free - 1] = 40
    pool.table[0, 0] = -1
    d, status = pool.dev(), i32([0])
    _, slots, positions = xqa.xqa_assign_pages(i32([2, 2]), d["lens"], d["table"], d["free"], d["num"], 4,
                                               status=status)
    assert slots.tolist() == [-1] * 4 and positions.tolist() == [10, 11, 16, 17]
    assert int(status) == xqa.XQA_ERR_BAD_BLOCK_ID and int(d["table"][1, 1]) == 40


def plain_release(pool, done):
    free, left, lens, errors = pool.free.copy(), pool.num_free, list(pool.ctx), set()
    for b, c in enumerate(pool.ctx):
        if not done[b]:
            continue
        lens[b] = 0
        if c < 0 or c > pool.mbs * 16:
            errors.add(xqa.XQA_ERR_CTX_TOO_LONG)
            continue
        for j in range((c + 15) // 16):
            if not 0 <= pool.table[b, j] < pool.nb:
                errors.add(xqa.XQA_ERR_BAD_BLOCK_ID)
            elif left == pool.nb:
                errors.add(xqa.XQA_ERR_NO_PAGES)
            else:
                free[left] = pool.table[b, j]
                left += 1
    return lens, free, left, errors


def check_release(pool, done, in_place=False, dtype=torch.bool):
    d, status = pool.dev(), i32([0])
    out = dict(new_lens=torch.full_like(d["lens"], 7), new_free=i32([7])) if not in_place else {}
    xqa.xqa_release_pages(torch.tensor(done).to(dtype).cuda(), d["lens"], d["table"], d["free"], d["num"],
                          status=status, **out)
    lens, free, left, errors = plain_release(pool, done)
    assert out.get("new_lens", d["lens"]).tolist() == lens
    assert out.get("new_free", d["num"]).tolist() == [left]
    assert np.array_equal(d["free"].cpu().numpy(), free)
    assert np.array_equal(d["table"].cpu().numpy(), pool.table)
    if not in_place:
        assert d["lens"].tolist() == pool.ctx and d["num"].tolist() == [pool.num_free]
    code = int(status)
    assert code in errors if errors else code == xqa.XQA_OK


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ctx,done", [([0], [1]), ([1], [1]), ([17], [0]), ([16, 17, 0, 40], [1, 0, 1, 1]),
                                      ([9000, 1, 8192, 8193], [1, 1, 1, 1])])
def test_small_releases(ctx, done, in_place):
    pool = Pool(ctx, 600, sum((c + 15) // 16 for c in ctx) + 7, seed=sum(ctx))
    check_release(pool, done, in_place, torch.uint8 if in_place else torch.bool)


@pytest.mark.parametrize("batch,reach", [(64, 100), (65, 3000), (700, 500), (1500, 40)])
def test_many_releases(batch, reach):
    g = np.random.default_rng(batch)
    ctx = [int(x) for x in g.integers(0, reach, batch)]
    done = [int(x) for x in g.integers(0, 2, batch)]
    pool = Pool(ctx, (reach + 15) // 16 + 600, sum((c + 15) // 16 for c in ctx) + 50, seed=batch)
    check_release(pool, done, in_place=bool(batch % 2))


def test_releases_with_errors():
    pool = Pool([40, 33, 100, 20], 9, 60)
    pool.table[0, 1] = 60
    pool.table[2, 3] = -1
    check_release(pool, [1, 1, 1, 1])
    pool.ctx[1] = 145
    check_release(pool, [1, 1, 0, 1], in_place=True)
    pool.ctx[1] = -1
    check_release(pool, [0, 1, 1, 0])
    full = Pool([40, 33], 9, 10)
    full.num_free = 8  # pages of the sequences are free already
    check_release(full, [1, 1])


def test_steps_in_a_graph_and_on_another_stream():
    """A page is with one sequence or free, never both, over many captured steps."""
    batch, mbs, nb = 40, 30, 700
    g = np.random.default_rng(1)
    lens, table = i32([0] * batch), torch.full((batch, mbs), -1, dtype=torch.int32, device="cuda")
    free, num = torch.randperm(nb).to(torch.int32).cuda(), i32([nb])
    new, done = i32([0] * batch), torch.zeros(batch, dtype=torch.bool, device="cuda")
    cu, slots, positions, status = i32([0] * (batch + 1)), i32([0] * 4000), i32([0] * 4000), i32([0])

    def step(stream=None):
        xqa.xqa_release_pages(done, lens, table, free, num, status=status, stream=stream)
        xqa.xqa_assign_pages(new, lens, table, free, num, 4000, cu_seqlens=cu, slots=slots,
                             positions=positions, status=status, stream=stream)

    step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(30):
        n = g.integers(0, 2 if i % 3 else 120, batch)
        d = g.random(batch) < 0.2
        before = [0 if e else c for c, e in zip(lens.tolist(), d)]
        n = [min(int(x), mbs * 16 - c) for x, c in zip(n, before)]
        new.copy_(i32(n))
        done.copy_(torch.from_numpy(d).cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = lens.tolist()
        assert got == [c + x for c, x in zip(before, n)] and int(status) == xqa.XQA_OK
        used = [int(table[b, j]) for b in range(batch) for j in range((got[b] + 15) // 16)]
        rest = free[:int(num)].tolist()
        assert sorted(used + rest) == list(range(nb))
        live = int(cu[-1])
        assert len(set(slots[:live].tolist())) == live and bool((slots[live:] == -1).all())


def test_binding_refusals():
    pool = Pool([10, 16], 5, 40)
    d = pool.dev()
    base = dict(new_tokens=i32([1, 1]), context_lens=d["lens"], block_tables=d["table"],
                free_pages=d["free"], num_free=d["num"], num_rows=4)
    for bad in (dict(new_tokens=i32([1])), dict(new_tokens=i32([1, 1]).cpu()), dict(num_rows=-1),
                dict(context_lens=d["lens"].long()), dict(block_tables=d["table"][:1]),
                dict(block_tables=d["table"].t()), dict(num_free=i32([1, 2])), dict(new_free=i32([])),
                dict(new_lens=i32([1])), dict(cu_seqlens=i32([0, 0])), dict(slots=i32([0])),
                dict(positions=i32([0] * 4).cpu()), dict(status=i32([0]).cpu())):
        with pytest.raises((ValueError, xqa.XqaError)):
            xqa.xqa_assign_pages(**{**base, **bad})
    done = torch.zeros(2, dtype=torch.bool, device="cuda")
    base = dict(done=done, context_lens=d["lens"], block_tables=d["table"], free_pages=d["free"],
                num_free=d["num"])
    for bad in (dict(done=done[:1]), dict(done=done.cpu()), dict(done=done.int()), dict(free_pages=d["free"].cpu()),
                dict(block_tables=d["table"][0]), dict(new_lens=i32([0]))):
        with pytest.raises((ValueError, xqa.XqaError)):
            xqa.xqa_release_pages(**{**base, **bad})
    assert d["lens"].tolist() == [10, 16]


def test_the_largest_batch():
    """16384 sequences, the most that shared memory holds, with and without a cluster."""
    batch = 16384
    for extra, rows in ((0, 2000), (6000, 30000)):
        g = np.random.default_rng(rows)
        ctx = g.integers(0, 33, batch)
        new = np.zeros(batch, np.int64)
        new[g.integers(0, batch, 900 + extra)] = 2
        pages = int(((ctx + new + 15) // 16).sum())
        pool = Pool([int(x) for x in ctx], 3, pages + 5, seed=rows)
        check_assign(pool, [int(x) for x in new], rows)
        check_release(pool, [int(x) for x in g.integers(0, 2, batch)])

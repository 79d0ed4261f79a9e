"""Measured cases of the operators around chunked and sparse serving.

Three sets that one serving step uses together: pages handed to requests as they grow and
taken back when they end (``xqa_assign_pages``, ``xqa_release_pages``), attention of a chunk
of new tokens over the paged cache (``xqa_extend``), and decode attention over the pages that
a cheap score selects (``xqa_page_bounds``, ``xqa_select``, ``xqa_decode_selected``). Each case
says what it stands for. Where ``own`` is false the operators run in plain torch operations;
where it is true, as the calls that a user makes.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128           # head dim
BS = 16           # tokens per page
BOUNDS = 272      # bytes of a (page, kv head) of the bounds: 128 upper, 128 lower, exponent, 15 zeros


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a few drafted tokens of one short sequence: latency
        dict(name="extend 1x5", op="extend", batch=1, min_new=5, max_new=5, min_ctx=705,
             max_ctx=705, hq=8, hkv=1, kv_dtype="e5m2", kv_layout="hnd", dtype="fp16",
             causal=True, lse=False, fused=False, k_scale=1.0, v_scale=1.0),
        # short turns of many long conversations
        dict(name="extend 16 short", op="extend", batch=16, min_new=2, max_new=32, min_ctx=4000,
             max_ctx=17000, hq=32, hkv=4, kv_dtype="e4m3", kv_layout="nhd", dtype="bf16",
             causal=True, lse=False, fused=True, k_scale=0.5, v_scale=0.25),
        # the next chunks of long prompts, q as a view of the projection, with the log-sum-exp
        dict(name="extend 4 chunks", op="extend", batch=4, min_new=1024, max_new=2048,
             min_ctx=6000, max_ctx=16384, hq=32, hkv=4, kv_dtype="e5m2", kv_layout="hnd",
             dtype="fp16", causal=True, lse=True, fused=True, k_scale=1.0, v_scale=1.0),
        # whole prompts, continuations and single tokens in one batch over a 4-bit cache
        dict(name="extend 4-bit ragged", op="extend", batch=9, min_new=1, max_new=600, min_ctx=600,
             max_ctx=8192, hq=24, hkv=8, kv_dtype="e2m1", kv_layout="hnd", dtype="bf16",
             causal=True, lse=False, fused=False, k_scale=0.5, v_scale=0.5),
        # the pages that a decode step's new tokens changed: latency
        dict(name="bounds 16 tokens", op="bounds", batch=16, min_new=1, max_new=1, min_ctx=2000,
             max_ctx=17800, hkv=4, kv_dtype="e4m3", kv_layout="nhd"),
        # the pages of long prompts
        dict(name="bounds 49k tokens", op="bounds", batch=4, min_new=9001, max_new=16384,
             min_ctx=9001, max_ctx=16384, hkv=4, kv_dtype="e5m2", kv_layout="hnd"),
        # the batch of long sequences of the framework's benchmark, 2048 tokens of each
        dict(name="sparse 16x17.8k", op="sparse", batch=16, min_ctx=16384, max_ctx=19200, hq=32,
             hkv=4, kv_dtype="e5m2", kv_layout="hnd", max_pages=128, first=1, last=2,
             k_scale=1.0, v_scale=1.0),
        # one very long sequence: most of the work is the choice
        dict(name="sparse 1x131k", op="sparse", batch=1, min_ctx=131072, max_ctx=131072, hq=32,
             hkv=8, kv_dtype="e4m3", kv_layout="nhd", max_pages=256, first=4, last=16,
             k_scale=0.5, v_scale=0.25),
        # a decode step: one token for each sequence, few need a page
        dict(name="assign 16x1", op="assign", batch=16, min_new=1, max_new=1, max_ctx=17800),
        # a mixed step of many requests: prompts, chunks, tokens and idle places
        dict(name="assign 512 ragged", op="assign", batch=512, min_new=0, max_new=512,
             max_ctx=16000),
        # two requests of a small batch end
        dict(name="release 2 of 16", op="release", batch=16, ending=2, max_ctx=17800),
        # many requests of a large batch end at once
        dict(name="release 200 of 512", op="release", batch=512, ending=200, max_ctx=16000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "extend", "extend", "bounds", "sparse", "sparse", "assign", "release"])
    if op in ("assign", "release"):
        batch, max_ctx = _log_int(rng, 1, 512), _log_int(rng, 1, 16000)
        if op == "release":
            return dict(op=op, batch=batch, ending=rng.randint(0, batch // 2 + 1) if batch > 1 else 1,
                        max_ctx=max_ctx)
        max_new = _log_int(rng, 1, 512)
        return dict(op=op, batch=batch, min_new=rng.randint(0, max_new), max_new=max_new,
                    max_ctx=max_ctx)
    kv_dtype = rng.choice(["e5m2", "e4m3", "e2m1"])
    case = dict(op=op, kv_dtype=kv_dtype,
                kv_layout="hnd" if kv_dtype == "e2m1" else rng.choice(["hnd", "nhd"]))
    if op == "bounds":
        max_ctx = _log_int(rng, 1, 16384)
        max_new = _log_int(rng, 1, max_ctx)
        case.update(batch=max(1, min(64, _log_int(rng, 1, 64), 60000 // max_ctx)),
                    min_new=rng.randint(1, max_new), max_new=max_new,
                    min_ctx=rng.randint(max_new, max_ctx), max_ctx=max_ctx,
                    hkv=rng.choice([1, 2, 4, 8]))
        return case
    hq, hkv = rng.choice([(8, 1), (32, 4), (32, 8), (16, 16), (24, 8), (12, 2), (16, 1), (20, 4)])
    case.update(hq=hq, hkv=hkv, k_scale=rng.choice([1.0, 0.5, 0.2937]),
                v_scale=rng.choice([1.0, 0.25, 0.7129]))
    if op == "sparse":
        max_ctx = _log_int(rng, 16, 65536)
        first, last = rng.randint(0, 4), rng.randint(1, 16)
        case.update(batch=max(1, min(64, _log_int(rng, 1, 64), 280000 // max_ctx)),
                    min_ctx=rng.randint(1, max_ctx), max_ctx=max_ctx, first=first, last=last,
                    max_pages=max(first + last, _log_int(rng, 4, 256)))
        return case
    max_ctx = _log_int(rng, 1, 16384)
    max_new = min(max_ctx, _log_int(rng, 1, 2048))
    batch = max(1, min(32, _log_int(rng, 1, 32), 200000 // max_ctx, 8000 // max_new))
    min_new = rng.randint(1, max_new)
    case.update(batch=batch, min_new=min_new, max_new=max_new,
                min_ctx=rng.randint(max_new, max_ctx), max_ctx=max_ctx,
                dtype=rng.choice(["fp16", "bf16"]), causal=rng.random() < 0.8,
                lse=rng.random() < 0.5, fused=rng.random() < 0.5)
    return case


def _ints(mix, n, lo, hi):
    """n whole numbers of [lo, hi], the largest among them."""
    r = random.Random(mix)
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _lengths(case):
    """(new tokens, tokens in all) of each sequence of a case: the same for every seed."""
    n = case["batch"]
    if case["op"] == "sparse":
        return [1] * n, _ints(3, n, case["min_ctx"], case["max_ctx"])
    if case["op"] == "assign":  # tokens before the step
        return _ints(4, n, case["min_new"], case["max_new"]), _ints(5, n, 0, case["max_ctx"])
    if case["op"] == "release":
        return [0] * n, _ints(6, n, 0, case["max_ctx"])
    new = _ints(1, n, case["min_new"], case["max_new"])
    return new, [max(a, b) for a, b in zip(new, _ints(2, n, case["min_ctx"], case["max_ctx"]))]


def _ending(case):
    return sorted(random.Random(7).sample(range(case["batch"]), min(case["batch"], case["ending"])))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.float16 if case.get("dtype", "fp16") == "fp16" else torch.bfloat16


def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _pages_of(tokens):
    return (tokens + BS - 1) // BS


def _tables(ctx, gen, width=0):
    """Block tables [B, MBS] (-1 behind a sequence) over a pool of pages in random order, the
    pool's size and its pages that no sequence has."""
    pages = [_pages_of(c) for c in ctx]
    total = sum(pages)
    nb = total + total // 4 + 1
    order = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(ctx), max(1, width, max(pages))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    return table, nb, order[at:]


def _pool(case, nb, gen):
    """A cache of normal values around each page's own, in the case's codes."""
    hkv = case["hkv"]
    hnd = case["kv_layout"] == "hnd"
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    x = rand(*((nb, hkv, BS, D) if hnd else (nb, BS, hkv, D)))
    x = (x + rand(*((nb, hkv, 1, D) if hnd else (nb, 1, hkv, D)))) * 0.7
    if case["kv_dtype"] == "e2m1":
        codes, scales = _quantise4(x)
        return torch.cat([codes.reshape(nb, hkv, -1), scales.reshape(nb, hkv, -1)], dim=2)
    return x.to(_float8(case["kv_dtype"])).view(torch.uint8)


def _quantise4(x):
    """x [..., 128] -> E2M1 codes [..., 64] and E4M3 scales [..., 8] (bytes)."""
    g = x.reshape(*x.shape[:-1], 8, 16)
    s8 = (g.abs().amax(dim=-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s8.float().unsqueeze(-1)
    a = torch.where(step > 0, g.abs() / step, torch.zeros_like(g))
    code = torch.signbit(g).to(torch.uint8) * 8
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += a > edge
    code = code.reshape(*x.shape[:-1], 64, 2)
    return code[..., 0] + 16 * code[..., 1], s8.view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new, ctx = _lengths(case)
    s = dict(case=case, new=new, ctx=ctx, lens=_i32(ctx))
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if case["op"] in ("assign", "release"):
        width = _pages_of(max(a + b for a, b in zip(new, ctx))) + 5
        s["table"], nb, free = _tables([a + b for a, b in zip(new, ctx)], gen, width)
        used = torch.arange(width, device="cuda") < _pages_of(s["lens"].long())[:, None]
        if case["op"] == "assign":  # the pages that this step will need are free still
            grow = torch.arange(width, device="cuda") < _pages_of((s["lens"] + _i32(new)).long())[:, None]
            free = torch.cat([free, s["table"][grow & ~used]])
            free = free[torch.randperm(free.numel(), generator=gen, device="cuda")]
            s["table"] = torch.where(used, s["table"], torch.full_like(s["table"], -1))
            s["new_tokens"], s["rows"] = _i32(new), sum(new) + 37
        else:
            s["done"] = torch.zeros(case["batch"], dtype=torch.bool)
            s["done"][_ending(case)] = True
            s["done"] = s["done"].cuda()
        s["free"] = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
        s["free"][:free.numel()] = free
        s["num_free"] = _i32([free.numel()])
        s["new_lens"], s["new_free"] = torch.empty_like(s["lens"]), torch.empty_like(s["num_free"])
        return s
    s["table"], nb, _ = _tables(ctx, gen)
    s["k_cache"] = _pool(case, nb, gen)
    if case["op"] != "sparse":
        s["cu"] = _offsets(new)
    if case["op"] == "bounds":
        s["bounds"] = torch.zeros((nb, case["hkv"], BOUNDS), dtype=torch.uint8, device="cuda")
        return s
    s["v_cache"] = _pool(case, nb, gen)
    s["k_scale"], s["v_scale"] = case["k_scale"], case["v_scale"]
    hq, hkv, t = case["hq"], case["hkv"], _dtype(case)
    if case["op"] == "sparse":
        s["q"] = rand(case["batch"], hq, D).to(t)
        s["bounds"] = torch.zeros((nb, hkv, BOUNDS), dtype=torch.uint8, device="cuda")
        for b, c in enumerate(ctx):  # as they stand after every step so far
            page = torch.arange(_pages_of(c), device="cuda")
            _plain_page_bounds(s, s["table"][b, :_pages_of(c)].long(), (c - page * BS).clamp(max=BS))
        return s
    if case["fused"]:
        s["q"] = rand(sum(new), hq + 2 * hkv, D).to(t)[:, :hq]
    else:
        s["q"] = rand(sum(new), hq, D).to(t)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"extend": _plain_extend, "bounds": _plain_bounds, "sparse": _plain_sparse,
            "assign": _plain_assign, "release": _plain_release}[s["case"]["op"]](s)


def _run_own(s):
    import paged_fp8_kv_gqa_gb300 as xqa

    case = s["case"]
    if case["op"] == "assign":
        cu, slots, positions = xqa.xqa_assign_pages(
            s["new_tokens"], s["lens"], s["table"], s["free"], s["num_free"], s["rows"],
            new_lens=s["new_lens"], new_free=s["new_free"])
        return s["new_lens"], s["table"], s["new_free"], cu, slots, positions
    if case["op"] == "release":
        xqa.xqa_release_pages(s["done"], s["lens"], s["table"], s["free"], s["num_free"],
                              new_lens=s["new_lens"], new_free=s["new_free"])
        return s["new_lens"], s["free"], s["new_free"]
    cache = dict(kv_dtype=case["kv_dtype"], kv_layout=case["kv_layout"])
    if case["op"] == "bounds":
        xqa.xqa_page_bounds(s["k_cache"], s["table"], s["lens"], s["cu"], sum(s["new"]), s["bounds"],
                            **cache)
        return s["bounds"].view(torch.int8)
    if case["op"] == "extend":
        if "shape" not in s:
            s["shape"] = xqa.make_extend_shape(s["q"], s["k_cache"], s["table"],
                                               causal=case["causal"], **cache)
            s["ws"] = xqa.alloc_extend_workspace(s["shape"], s["q"].device)
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if case["lse"] else None
        out = xqa.xqa_extend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                             s["k_scale"], s["v_scale"], lse=lse, workspace=s["ws"],
                             shape=s["shape"])
        return (out, lse) if case["lse"] else out
    if "shape" not in s:
        s["choice"] = xqa.make_select_shape(s["q"], s["bounds"], s["table"], case["max_pages"],
                                            case["first"], case["last"])
        s["choice_ws"] = xqa.alloc_select_workspace(s["choice"], s["q"].device)
    selected, lens = xqa.xqa_select(s["q"], s["bounds"], s["table"], s["lens"],
                                    workspace=s["choice_ws"], shape=s["choice"])
    if "shape" not in s:
        s["shape"] = xqa.make_selected_shape(s["q"], s["k_cache"], selected, **cache)
        s["ws"] = xqa.alloc_workspace(s["shape"], s["q"].device)
    out = xqa.xqa_decode_selected(s["q"], s["k_cache"], s["v_cache"], selected, lens, s["k_scale"],
                                  s["v_scale"], workspace=s["ws"], shape=s["shape"])
    return out, selected, lens


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e in 32 bits of whole numbers e (as the bits say it: a power function may round)."""
    return ((e.to(torch.int32).clamp(-126, 127) + 127) << 23).view(torch.float32)


def _float8(kv_dtype):
    return torch.float8_e5m2 if kv_dtype == "e5m2" else torch.float8_e4m3fn


def _decode4(codes, scales):
    """The values of codes [..., 64] and scales [..., 8]: [..., 128] in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0,
                          -3.0, -4.0, -6.0], device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*codes.shape[:-1], 8, 16)
    val = table[nib.long()] * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return val.reshape(*codes.shape[:-1], 128)


def _page_values(case, cache, pages):
    """Values in 32 bits of whole pages: [..., BS, hkv, 128], before the tensor's scale."""
    x = cache[pages]
    if case["kv_dtype"] == "e2m1":
        codes, scales = x[..., :1024].unflatten(-1, (BS, 64)), x[..., 1024:].unflatten(-1, (BS, 8))
        return _decode4(codes, scales).transpose(-2, -3)
    x = x.view(_float8(case["kv_dtype"])).float()
    return x.transpose(-2, -3) if case["kv_layout"] == "hnd" else x


def _plain_extend(s):
    case = s["case"]
    hq, hkv, g = case["hq"], case["hkv"], case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float32, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float32, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(s["new"], s["ctx"])):
        pages = s["table"][b, :_pages_of(c)].long()
        k = _page_values(case, s["k_cache"], pages).reshape(-1, hkv, D)[:c].permute(1, 2, 0)
        v = _page_values(case, s["v_cache"], pages).reshape(-1, hkv, D)[:c].transpose(0, 1)
        q = s["q"][at:at + n].float().view(n, hkv, g, D).permute(1, 2, 0, 3).reshape(hkv, g * n, D)
        sc = torch.matmul(q, k).mul_(s["k_scale"] / math.sqrt(D)).view(hkv, g, n, c)
        if case["causal"]:
            i, t = torch.arange(n, device="cuda"), torch.arange(c, device="cuda")
            sc.masked_fill_(t > (c - n + i)[:, None], -math.inf)
        m = sc.amax(dim=-1, keepdim=True)
        p = sc.sub_(m).exp_()
        tot = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.view(hkv, g * n, c), v).view(hkv, g, n, D) / tot * s["v_scale"]
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, D)
        lse[at:at + n] = (m + tot.log()).squeeze(-1).permute(2, 0, 1).reshape(n, hq)
        at += n
    out = out.to(s["q"].dtype)
    return (out, lse) if case["lse"] else out


def _plain_page_bounds(s, pages, fill):
    """Writes the bounds of pages of which the first ``fill`` tokens are in use."""
    x = _page_values(s["case"], s["k_cache"], pages)                     # [n, BS, hkv, D]
    used = (torch.arange(BS, device="cuda") < fill[:, None])[:, :, None, None]
    x = torch.where(used, x, torch.zeros_like(x))
    finite = torch.isfinite(x).all(dim=-1).all(dim=1)                    # [n, hkv]
    x = torch.where(finite[:, None, :, None], x, torch.zeros_like(x))
    low = torch.where(used, x, torch.full_like(x, math.inf)).amin(dim=1)
    high = torch.where(used, x, torch.full_like(x, -math.inf)).amax(dim=1)
    top = torch.maximum(high.abs(), low.abs()).amax(dim=-1)              # [n, hkv]
    # 2^(e + 6) <= top < 2^(e + 7): top is at most 127 steps of 2^e
    e = torch.where(top > 0, torch.frexp(top).exponent - 7, torch.zeros_like(top, dtype=torch.int32))
    step = _pow2(-e)[..., None]
    res = torch.zeros((pages.numel(), s["case"]["hkv"], BOUNDS), dtype=torch.int8, device="cuda")
    res[..., :D] = torch.ceil(high * step).to(torch.int8)
    res[..., D:2 * D] = torch.floor(low * step).to(torch.int8)
    res[..., 2 * D] = torch.where(finite, e, torch.full_like(e, -128)).to(torch.int8)
    s["bounds"][pages] = res.view(torch.uint8)


def _plain_bounds(s):
    pages, fill = [], []
    for b, (n, c) in enumerate(zip(s["new"], s["ctx"])):
        page = torch.arange((c - n) // BS, _pages_of(c), device="cuda")
        pages.append(s["table"][b, (c - n) // BS:_pages_of(c)])
        fill.append(c - page * BS)
    _plain_page_bounds(s, torch.cat(pages).long(), torch.cat(fill).clamp(max=BS))
    return s["bounds"].view(torch.int8)


def _plain_sparse(s):
    case = s["case"]
    b, hq, hkv, g, top = case["batch"], case["hq"], case["hkv"], case["hq"] // case["hkv"], case["max_pages"]
    lens = s["lens"].long()
    num = _pages_of(lens)
    nmax = max(_pages_of(c) for c in s["ctx"])
    # the group's query in whole steps, its positive and negative part over the heads
    q = s["q"].float().view(b, hkv, g, D)
    e = torch.frexp(q.abs().amax(dim=(2, 3))).exponent - 6
    q8 = torch.round(q * _pow2(-e)[:, :, None, None])
    up, down = q8.clamp(min=0).sum(dim=2), q8.clamp(max=0).sum(dim=2)    # [b, hkv, D]
    pages = s["table"].long()[:, :nmax]
    bd = s["bounds"].view(torch.int8)[pages.clamp(min=0)].float()        # [b, nmax, hkv, 272]
    score = torch.einsum("bhd,bphd->bhp", up, bd[..., :D]) + torch.einsum("bhd,bphd->bhp", down, bd[..., D:2 * D])
    exp = bd[..., 2 * D].transpose(1, 2)
    score = (score * _pow2(exp)).masked_fill(exp == -128, 1e37)
    j = torch.arange(nmax, device="cuda")
    always = (j < case["first"]) | (j >= (num - case["last"])[:, None])
    score = score.masked_fill(always[:, None], 2e37).masked_fill((j >= num[:, None])[:, None], -2e37)
    keep = min(top, nmax)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    take = torch.minimum(num, torch.full_like(num, top))                 # [b]
    k = torch.arange(keep, device="cuda")
    order = torch.where(k < take[:, None, None], order, torch.full_like(order, nmax)).sort(dim=-1).values
    some = k < take[:, None, None]
    phys = torch.gather(pages[:, None].expand(b, hkv, nmax), 2, order.clamp(max=nmax - 1))
    selected = torch.full((b, hkv, top), -1, dtype=torch.int32, device="cuda")
    selected[..., :keep] = torch.where(some, phys, torch.full_like(phys, -1)).to(torch.int32)
    sel_lens = (lens - (num - take) * BS)[:, None].expand(b, hkv).to(torch.int32).contiguous()
    # attention over them
    head = torch.arange(hkv, device="cuda")[None, :, None].expand(b, hkv, keep)
    at = phys.clamp(min=0)

    def values(cache):
        if case["kv_dtype"] == "e2m1":
            x = cache[at, head]
            return _decode4(x[..., :1024].unflatten(-1, (BS, 64)), x[..., 1024:].unflatten(-1, (BS, 8)))
        x = cache[at, head] if case["kv_layout"] == "hnd" else cache[at, :, head]
        return x.view(_float8(case["kv_dtype"])).float()

    kk = values(s["k_cache"]).reshape(b, hkv, keep * BS, D)
    vv = values(s["v_cache"]).reshape(b, hkv, keep * BS, D)
    sc = torch.matmul(q, kk.transpose(-1, -2)) * (s["k_scale"] / math.sqrt(D))
    sc = sc.masked_fill((torch.arange(keep * BS, device="cuda") >= sel_lens[..., None])[:, :, None], -math.inf)
    p = (sc - sc.amax(dim=-1, keepdim=True)).exp()
    out = torch.matmul(p, vv) / p.sum(dim=-1, keepdim=True) * s["v_scale"]
    return out.view(b, hq, D).to(s["q"].dtype), selected, sel_lens


def _plain_assign(s):
    table, rows = s["table"], s["rows"]
    n, old, free = s["new_tokens"].long(), s["lens"].long(), s["num_free"].long()
    ok = (n >= 0) & (old >= 0) & (old + n <= table.shape[1] * BS)
    n = torch.where(ok, n, torch.zeros_like(n))
    n = torch.where(n.cumsum(0) <= rows, n, torch.zeros_like(n))
    need = _pages_of(old + n) - _pages_of(old)
    upto = need.cumsum(0)
    n = torch.where((need == 0) | (upto <= free), n, torch.zeros_like(n))
    lens = old + n
    first, pages = _pages_of(old), _pages_of(lens)
    j = torch.arange(table.shape[1], device="cuda")
    fresh = (j >= first[:, None]) & (j < pages[:, None])
    rank = (upto - need)[:, None] + j - first[:, None]
    got = s["free"][(free - 1 - rank).clamp(min=0, max=s["free"].numel() - 1)]
    table.copy_(torch.where(fresh, got, table))
    cu = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    r = torch.arange(rows, device="cuda")
    b = torch.bucketize(r, cu[1:], right=True)
    some = b < n.numel()
    b = b.clamp(max=n.numel() - 1)
    pos = old[b] + r - cu[b]
    slot = table.long()[b, (pos // BS).clamp(max=table.shape[1] - 1)] * BS + pos % BS
    none = torch.full_like(pos, -1)
    left = free - torch.where(pages > first, upto, torch.zeros_like(upto)).amax()
    return (lens.to(torch.int32), table, left.to(torch.int32), cu.to(torch.int32),
            torch.where(some, slot, none).to(torch.int32), torch.where(some, pos, none).to(torch.int32))


def _plain_release(s):
    table, lens, free = s["table"], s["lens"].long(), s["free"]
    j = torch.arange(table.shape[1], device="cuda")
    back = s["done"][:, None] & (j < _pages_of(lens)[:, None]) & (table >= 0) & (table < free.numel())
    upto = back.reshape(-1).long().cumsum(0)
    at = s["num_free"].long() + upto - 1
    at = torch.where(back.reshape(-1) & (at < free.numel()), at, torch.full_like(at, free.numel()))
    longer = torch.cat([free, free[:1]])
    longer[at] = table.reshape(-1)
    free.copy_(longer[:-1])
    left = (s["num_free"].long() + upto[-1]).clamp(max=free.numel())
    return torch.where(s["done"], torch.zeros_like(s["lens"]), s["lens"]), free, left.to(torch.int32)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    new, ctx = _lengths(case)
    b = case["batch"]
    if case["op"] == "assign":
        pages = sum(_pages_of(n + c) - _pages_of(c) for n, c in zip(new, ctx))
        return {"bytes": 4 * (4 * b + 2 + 2 * pages + 2 * sum(new)), "flops": sum(new)}
    if case["op"] == "release":
        pages = sum(_pages_of(ctx[i]) for i in _ending(case))
        return {"bytes": 9 * b + 8 + 8 * pages, "flops": pages}
    token = 72 if case["kv_dtype"] == "e2m1" else 128
    hkv = case["hkv"]
    if case["op"] == "bounds":
        pages = sum(_pages_of(c) - (c - n) // BS for n, c in zip(new, ctx))
        tokens = sum(c - (c - n) // BS * BS for n, c in zip(new, ctx))
        return {"bytes": hkv * (pages * BOUNDS + tokens * token), "flops": 2 * D * hkv * tokens}
    hq = case["hq"]
    if case["op"] == "sparse":
        read = sum(min(c, c - (_pages_of(c) - case["max_pages"]) * BS) for c in ctx)
        pages = sum(_pages_of(c) for c in ctx if _pages_of(c) > case["max_pages"])
        return {"bytes": hkv * (2 * token * read + (2 * D + 1) * pages) + 4 * D * hq * b
                + 4 * hkv * sum(min(_pages_of(c), case["max_pages"]) for c in ctx),
                "flops": 4 * D * hq * read + 4 * D * hkv * pages}
    nbytes = 2 * token * hkv * sum(ctx) + 4 * D * hq * sum(new) + (4 * hq * sum(new) if case["lse"] else 0)
    pairs = sum(n * c - (n * (n - 1) // 2 if case["causal"] else 0) for n, c in zip(new, ctx))
    return {"bytes": nbytes, "flops": 4 * D * hq * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "bounds": _exact_bounds, "sparse": _exact_sparse,
            "assign": _exact_assign, "release": _exact_release}[case["op"]](s)


def _code_values(kv_dtype):
    """The 256 codes' values in 64 bits, from the formats' definitions."""
    man, bias = (2, 15) if kv_dtype == "e5m2" else (3, 7)
    vals = []
    for c in range(256):
        e, f = (c & 127) >> man, c & ((1 << man) - 1)
        x = f * 2.0 ** (1 - bias - man) if e == 0 else (1 + f / (1 << man)) * 2.0 ** (e - bias)
        if kv_dtype == "e5m2" and e == 31:
            x = math.inf if f == 0 else math.nan
        if kv_dtype != "e5m2" and c & 127 == 127:
            x = math.nan
        vals.append(-x if c & 128 else x)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _exact_tokens(case, cache, pages, n, h):
    """The values in 64 bits, before the tensor's scale, of kv head h's first n tokens: [n, 128]."""
    if case["kv_dtype"] != "e2m1":
        x = cache[pages.long()][:, h] if case["kv_layout"] == "hnd" else cache[pages.long()][:, :, h]
        return _code_values(case["kv_dtype"])[x.long()].reshape(-1, D)[:n]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                        dtype=torch.float64, device="cuda")
    x = cache[pages.long()][:, h].long()
    codes = x[:, :1024].reshape(-1, 64)[:n]
    scale = _code_values("e4m3")[x[:, 1024:].reshape(-1, 8)[:n]]
    out = torch.empty((n, D), dtype=torch.float64, device="cuda")
    out[:, 0::2], out[:, 1::2] = grid[codes % 16], grid[codes // 16]
    return (out.view(n, 8, 16) * scale[..., None]).view(n, D)


def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale64(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _exact_extend(s):
    case = s["case"]
    hq, hkv = case["hq"], case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(s["new"], s["ctx"])):
        pages = s["table"][b, :_pages_of(c)]
        hidden = torch.ones((n, c), dtype=torch.bool, device="cuda").triu(c - n + 1) if case["causal"] else None
        for h in range(hq):
            if h % (hq // hkv) == 0:
                k = _exact_tokens(case, s["k_cache"], pages, c, h * hkv // hq) * _scale64(s["k_scale"])
                v = _exact_tokens(case, s["v_cache"], pages, c, h * hkv // hq) * _scale64(s["v_scale"])
            sc = s["q"][at:at + n, h].double() @ k.T / math.sqrt(D)
            if hidden is not None:
                sc.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(sc, dim=-1)
            lse[at:at + n, h] = z
            out[at:at + n, h] = sc.sub_(z[:, None]).exp_() @ v
        at += n
    return (out, lse) if case["lse"] else out


def _exact_bounds(s):
    case = s["case"]
    res = s["bounds"].view(torch.int8).clone()
    for b, (n, c) in enumerate(zip(s["new"], s["ctx"])):
        first = (c - n) // BS
        for h in range(case["hkv"]):
            pages = s["table"][b, first:_pages_of(c)]
            x = _exact_tokens(case, s["k_cache"], pages, c - first * BS, h)
            pad = torch.cat([x, x[-1:].expand(-x.shape[0] % BS, D)]).view(-1, BS, D)
            high, low = pad.amax(dim=1), pad.amin(dim=1)
            top = torch.maximum(high, -low).amax(dim=1)
            e = torch.where(top > 0, torch.floor(torch.log2(top)) - 6, torch.zeros_like(top))
            row = torch.zeros((pages.numel(), BOUNDS), dtype=torch.float64, device="cuda")
            row[:, :D] = torch.ceil(high / _pow2_64(e)[:, None])
            row[:, D:2 * D] = torch.floor(low / _pow2_64(e)[:, None])
            row[:, 2 * D] = e
            res[pages.long(), h] = row.to(torch.int8)
    return res


def _exact_sparse(s):
    case = s["case"]
    hq, hkv, g, top = case["hq"], case["hkv"], case["hq"] // case["hkv"], case["max_pages"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    selected = torch.full((case["batch"], hkv, top), -1, dtype=torch.int32)
    lens = torch.zeros((case["batch"], hkv), dtype=torch.int32)
    for b, c in enumerate(s["ctx"]):
        num = _pages_of(c)
        pages = s["table"][b, :num]
        for h in range(hkv):
            q = s["q"][b, h * g:(h + 1) * g].double()
            step = _pow2_64(torch.floor(torch.log2(q.abs().max())) - 5)
            w = torch.round(q / step)
            bd = s["bounds"].view(torch.int8)[pages.long(), h].double()
            score = bd[:, :D] @ w.clamp(min=0).sum(0) + bd[:, D:2 * D] @ w.clamp(max=0).sum(0)
            score = (score * _pow2_64(bd[:, 2 * D])).tolist()
            forced = [j for j in range(num) if j < case["first"] or j >= num - case["last"]]
            rest = sorted((j for j in range(case["first"], max(case["first"], num - case["last"]))),
                          key=lambda j: (-score[j], j))
            take = sorted((forced + rest)[:top])
            chosen = pages.cpu()[torch.tensor(take)]
            selected[b, h, :len(take)] = chosen
            n = c - (num - len(take)) * BS
            lens[b, h] = n
            k = _exact_tokens(case, s["k_cache"], chosen.cuda(), n, h) * _scale64(s["k_scale"])
            v = _exact_tokens(case, s["v_cache"], chosen.cuda(), n, h) * _scale64(s["v_scale"])
            out[b, h * g:(h + 1) * g] = torch.softmax(q @ k.T / math.sqrt(D), dim=-1) @ v
    return out, selected.cuda(), lens.cuda()


def _exact_assign(s):
    """One request after another, as the definition says it."""
    table, free = s["table"].cpu().tolist(), s["free"].cpu().tolist()
    left, rows = int(s["num_free"]), s["rows"]
    cu, slots, positions, lens = [0], [], [], []
    for b, (n, c) in enumerate(zip(s["new"], s["ctx"])):
        for pos in range(c, c + n):
            if pos % BS == 0:
                left -= 1
                table[b][pos // BS] = free[left]
            slots.append(table[b][pos // BS] * BS + pos % BS)
            positions.append(pos)
        cu.append(cu[-1] + n)
        lens.append(c + n)
    pad = [-1] * (rows - len(slots))
    return tuple(_i32(x) for x in (lens, table, [left], cu, slots + pad, positions + pad))


def _exact_release(s):
    table, free, left = s["table"].cpu().tolist(), s["free"].cpu().tolist(), int(s["num_free"])
    lens = list(s["ctx"])
    for b in _ending(s["case"]):
        for j in range(_pages_of(lens[b])):
            free[left] = table[b][j]
            left += 1
        lens[b] = 0
    return _i32(lens), _i32(free), _i32([left])

"""Measured cases of the block-scaled per-head cache: page tables built from request lengths,
the append that quantises each block of tokens and head with a scale of its own, the gather of
cached positions into packed rows, and the attention of a request's newest tokens.

Every case is a dict of plain values.  ``run`` makes one pass through an operator, in the
plain form (elementary torch operations in fp32) where ``own`` is false and through the
library's entry points where it is true.  ``exact`` computes the same outputs from the
definition in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
MAX_POS = 73728            # rows of the rotary table


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # The tables of one decode step of 64 conversations: the smallest call, launch alone.
        dict(name="table_step", op="table", requests=64, shortest=1, longest=1, context=65535, mix=1,
             page=128, idle=0),
        # 24 conversations on one-token pages, each behind 63,911 cached positions with 4,089 new
        # ones: every new token takes a page.
        dict(name="table_prompts", op="table", requests=24, shortest=4089, longest=4089, context=63911,
             mix=2, page=1, idle=0),
        # One decode step of 64 requests on a two-KV-head shard: one new row in a block that
        # others started.
        dict(name="append_step", op="append", requests=64, shortest=1, longest=1, context=4089, mix=3,
             q_heads=16, kv_heads=2, dim=128, rot=128, neox=True, page=128, block=128, k_out=False, idle=0),
        # Fresh prompts of 16,384 tokens in all, the rotated keys kept for the prompt's attention.
        dict(name="append_prompts", op="append", requests=4, shortest=4096, longest=4096, context=0, mix=4,
             q_heads=32, kv_heads=8, dim=128, rot=128, neox=True, page=128, block=64, k_out=True, idle=0),
        # Ragged chunks behind short contexts, 64-wide heads of which 32 columns rotate in
        # interleaved pairs, five query heads a KV head, small pages, some idle requests.
        dict(name="append_chunks", op="append", requests=37, shortest=1, longest=700, context=300, mix=5,
             q_heads=25, kv_heads=5, dim=64, rot=32, neox=False, page=16, block=16, k_out=True, idle=7),
        # A question of 4,089 tokens behind a prefix of 63,911 that the cache holds: its keys and
        # values as packed rows for the prompt's attention.
        dict(name="gather_prefix", op="gather", requests=1, shortest=4089, longest=4089, context=63911,
             fixed=True, mix=6, kv_heads=8, dim=128, page=128, block=128, idle=0),
        # Ragged short prompts, 64-wide heads, small pages.
        dict(name="gather_ragged", op="gather", requests=53, shortest=1, longest=700, context=300,
             fixed=False, mix=7, kv_heads=2, dim=64, page=16, block=16, idle=9),
        # One request with a short history: latency alone.
        dict(name="decode_short", op="decode", requests=1, shortest=137, longest=137, new=1, mix=8,
             q_heads=32, kv_heads=8, dim=128, page=16, block=16, idle=0),
        # A serving batch: 64 requests of 2,048 .. 65,536 positions, a two-KV-head shard.
        dict(name="decode_batch", op="decode", requests=64, shortest=2048, longest=65536, new=1, mix=9,
             q_heads=16, kv_heads=2, dim=128, page=128, block=128, idle=0),
        # One conversation of 142,000 positions: split over its length.
        dict(name="decode_long", op="decode", requests=1, shortest=142000, longest=142000, new=1, mix=10,
             q_heads=64, kv_heads=8, dim=128, page=128, block=64, idle=0),
        # Ragged lengths, five query heads a KV head, 64-wide heads, small pages, idle slots.
        dict(name="decode_ragged", op="decode", requests=37, shortest=1, longest=4089, new=1, mix=11,
             q_heads=20, kv_heads=4, dim=64, page=16, block=16, idle=10),
        # Four draft tokens of each of 64 requests verified at once, 32 query rows a KV head.
        dict(name="decode_verify", op="decode", requests=64, shortest=2048, longest=65536, new=4, mix=12,
             q_heads=16, kv_heads=2, dim=128, page=128, block=128, idle=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    """What bounds a drawn case: bytes, flops, and the elements of the plain form's padded caches."""
    w = work(case)
    if case["op"] != "decode":
        return w["bytes"], w["flops"], 0
    return w["bytes"], w["flops"], case["requests"] * max(_lengths(case)[1]) * case["kv_heads"] * case["dim"]


def draw(rng):
    """One more case of the listed ranges, no dearer than the largest listed one."""
    largest = {}
    for c in listed():
        old = largest.get(c["op"], (0, 0, 0))
        largest[c["op"]] = tuple(max(a, b) for a, b in zip(old, _cost(c)))
    while True:
        op = rng.choice(("table", "append", "gather", "decode", "decode"))
        page = rng.choice((1, 16, 32, 64, 128))
        case = dict(op=op, requests=_log_int(rng, 1, 256), mix=rng.randrange(1, 10 ** 6), page=page,
                    idle=rng.choice((0, 0, 5, 10)))
        if op == "decode":
            longest = _log_int(rng, 1, 142000)
            case.update(longest=longest, shortest=_log_int(rng, 1, longest), new=rng.choice((1, 1, 1, 2, 3, 4, 8)))
        else:
            longest = _log_int(rng, 1, 16384)
            case.update(longest=longest, shortest=_log_int(rng, 1, longest),
                        context=rng.choice((0, _log_int(rng, 1, 65535 if op != "append" else 4089))))
            if op == "gather":
                case.update(fixed=rng.random() < 0.5)
        if op != "table":
            dim = rng.choice((64, 128))
            kv_heads = rng.choice((1, 2, 3, 4, 5, 8))
            case.update(kv_heads=kv_heads, dim=dim, block=rng.choice([b for b in (1, 4, 16, 32, 64, 128) if b <= page]))
            if op != "gather":
                case.update(q_heads=kv_heads * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16)))
            if op == "append":
                case.update(rot=rng.choice([r for r in (16, 32, 64, 96, 128) if r <= dim]),
                            neox=rng.random() < 0.5, k_out=rng.random() < 0.5)
        if all(a <= b for a, b in zip(_cost(case), largest[op])):
            return case


def _lengths(case):
    """(new tokens, positions) of every request, the longest among them; every idle-th request
    has none.  A property of the case, not of the seed."""
    rng = random.Random(case["mix"])
    n = case["requests"]
    some = [_log_int(rng, case["shortest"], case["longest"]) for _ in range(n)]
    some[rng.randrange(n)] = case["longest"]
    if case["op"] == "decode":
        held = [0 if case["idle"] and b % case["idle"] == case["idle"] - 1 else x for b, x in enumerate(some)]
        return [case["new"]] * n, held
    if case.get("fixed"):
        before = [case["context"]] * n
    else:
        before = [rng.randrange(0, case["context"] + 1) for _ in range(n)]
    for b in range(n):
        if case["idle"] and b % case["idle"] == case["idle"] - 1:
            some[b] = before[b] = 0
    return some, [x + c for x, c in zip(some, before)]


def _pages(case, held):
    return [-(-x // case["page"]) for x in held]


def work(case):
    new, held = _lengths(case)
    n, pages, total = len(held), sum(_pages(case, held)), sum(held)
    if case["op"] == "table":
        taken = pages - sum(-(-(x - t) // case["page"]) for t, x in zip(new, held))
        return {"bytes": 4 * (2 * n + 3 * (n + 1) + n) + 8 * (pages - taken) + 12 * taken + 8 * sum(new),
                "flops": 0}
    hk, d = case["kv_heads"], case["dim"]
    lists = 4 * (pages + 3 * n + 2)
    blocks = sum(-(-x // case["block"]) for x in held)
    if case["op"] == "gather":
        cached = total - sum(new)
        return {"bytes": 2 * hk * d * (cached + 2 * total + 2 * sum(new)) + 8 * hk * blocks + lists,
                "flops": 2 * hk * d * cached}
    hq = case["q_heads"]
    if case["op"] == "append":
        t = sum(new)
        return {"bytes": t * (hq * d * 4 + 2 * hk * d * 3 + (2 * hk * d if case["k_out"] else 0) + 4 + 4 * case["rot"])
                         + 8 * hk * min(blocks, t) + lists,
                "flops": 3 * t * (hq + hk) * case["rot"]}
    return {"bytes": 2 * hk * d * total + 8 * hk * blocks + sum(new) * hq * (4 * d + 4) + lists,
            "flops": 4 * hq * d * sum(t * x - t * (t - 1) // 2 for t, x in zip(new, held) if x >= t)}


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    """N(0, std^2), made in slices so that large tensors need no fp32 copy."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device=DEV) * std
        flat[i:i + n] = x.clamp_(-448, 448).to(dtype)
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _sums(counts):
    out = [0]
    for x in counts:
        out.append(out[-1] + x)
    return _ints(out)


def _paged(case, g, held):
    """The page table of requests with `held` positions, over a pool with some pages to spare."""
    pages = _pages(case, held)
    total = sum(pages)
    pool = total + max(1, total // 16)
    return dict(pool=pool, kv_indptr=_sums(pages),
                kv_indices=torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32),
                kv_last_page_lens=_ints([max(1, x - (p - 1) * case["page"]) for x, p in zip(held, pages)]))


def _cache(case, g, pool):
    """Codes and their blocks' scales, as the append leaves them (powers of two)."""
    shape = (pool, case["page"], case["kv_heads"], case["dim"])
    blocks = (pool, case["page"] // case["block"], case["kv_heads"])
    scale = lambda lo: torch.exp2(torch.randint(lo, lo + 3, blocks, generator=g, device=DEV).float())
    return dict(k_cache=_normal(g, shape, 100.0, torch.float8_e4m3fn), k_scale=scale(-8),
                v_cache=_normal(g, shape, 100.0, torch.float8_e4m3fn), v_scale=scale(-9))


def _table_inputs(case, seed):
    g = _gen(seed)
    new, held = _lengths(case)
    pages = _pages(case, held)
    most = max(1, max(pages))
    had = [-(-(x - t) // case["page"]) for t, x in zip(new, held)]
    pool = sum(pages) + 8
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(held), most), -1, dtype=torch.int32, device=DEV)
    b = torch.arange(len(held), device=DEV).repeat_interleave(_ints(had).long())
    at = torch.arange(sum(had), device=DEV)
    table[b, at - _sums(had).long()[b]] = ids[:sum(had)]
    empty = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)
    n = len(held)
    return dict(case=case, seq_lens=_ints(held), new_lens=_ints(new), block_table=table,
                free_pages=ids[sum(had):].clone(), free_count=_ints([pool - sum(had)]),
                free_count_out=empty(1), qo_indptr=empty(n + 1), key_indptr=empty(n + 1),
                kv_indptr=empty(n + 1), kv_indices=torch.zeros(sum(pages) + 64, dtype=torch.int32, device=DEV),
                kv_last_page_lens=empty(n), positions=empty(sum(new) + 5), slots=empty(sum(new) + 5),
                error_word=torch.zeros(2, dtype=torch.int32, device=DEV))


def _append_inputs(case, seed):
    g = _gen(seed)
    hq, hk, d, r = (case[k] for k in ("q_heads", "kv_heads", "dim", "rot"))
    new, held = _lengths(case)
    t = sum(new)
    st = dict(case=case, qo_indptr=_sums(new), **_paged(case, g, held))
    st.update(_cache(case, g, st["pool"]))
    # rows whose sizes differ, so that later rows grow a block's scale now and then
    spread = torch.exp2(torch.randn(t, 1, 1, generator=g, device=DEV))
    st["q"] = _normal(g, (t, hq, d))
    st["k"] = (_normal(g, (t, hk, d)) * spread).to(torch.bfloat16)
    st["v"] = (_normal(g, (t, hk, d)) * spread).to(torch.bfloat16)
    st["positions"] = torch.randint(0, MAX_POS, (t,), generator=g, device=DEV, dtype=torch.int32)
    # the rotary table of a serving engine: fp32 cosines and sines, the angles in fp64
    inv = 10000.0 ** (-torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / r)
    ang = torch.arange(MAX_POS, device=DEV, dtype=torch.float64)[:, None] * inv
    st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    st["q_out"] = torch.empty_like(st["q"])
    st["k_out"] = torch.empty_like(st["k"]) if case["k_out"] else None
    st["error_word"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def _gather_inputs(case, seed):
    g = _gen(seed)
    hk, d = case["kv_heads"], case["dim"]
    new, held = _lengths(case)
    st = dict(case=case, qo_indptr=_sums(new), key_indptr=_sums(held), **_paged(case, g, held))
    st.update(_cache(case, g, st["pool"]))
    st["k_new"] = _normal(g, (sum(new), hk, d))
    st["v_new"] = _normal(g, (sum(new), hk, d))
    st["k_rows"] = torch.zeros((sum(held) + 3, hk, d), dtype=torch.bfloat16, device=DEV)
    st["v_rows"] = torch.zeros((sum(held) + 3, hk, d), dtype=torch.bfloat16, device=DEV)
    st["error_word"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def _decode_inputs(case, seed):
    g = _gen(seed)
    hq, d = case["q_heads"], case["dim"]
    new, held = _lengths(case)
    st = dict(case=case, qo_indptr=_sums(new), **_paged(case, g, held))
    st.update(_cache(case, g, st["pool"]))
    st["q"] = _normal(g, (sum(new), hq, d), 1.5)
    st["sm_scale"] = d ** -0.5
    st["o"] = torch.empty((sum(new), hq, d), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty((sum(new), hq), dtype=torch.float32, device=DEV)
    return st


_INPUTS = {"table": _table_inputs, "append": _append_inputs, "gather": _gather_inputs, "decode": _decode_inputs}


def prepare(case, seed):
    st = _INPUTS[case["op"]](case, seed)
    if own and case["op"] == "decode":
        import paged_mla_latent_gb300 as pm
        st["workspace"] = pm.make_gqa_block_decode_workspace(case["q_heads"], case["kv_heads"],
                                                             case["dim"], case["new"], DEV)
    return st


# ----------------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _running(counts):
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])


def _owner(start, n):
    """The request of each of n entries whose requests start at start[:-1] (empty ones skipped);
    entries past the end get the last request."""
    i = torch.arange(n, device=DEV)
    return i, torch.searchsorted(start[1:].contiguous(), i, right=True).clamp_(max=start.numel() - 2)


def _plain_table(st):
    ps = st["case"]["page"]
    held, new = st["seq_lens"].long(), st["new_lens"].long()
    pages = (held + ps - 1) // ps
    had = (held - new + ps - 1) // ps
    taken, kv, qo = _running(pages - had), _running(pages), _running(new)
    table, free = st["block_table"], st["free_pages"]
    column = torch.arange(table.shape[1], device=DEV)[None, :]
    nth = taken[:-1, None] + column - had[:, None]
    page = free[(st["free_count"].long() - 1 - nth).clamp(0, free.numel() - 1)]
    table.copy_(torch.where((column >= had[:, None]) & (column < pages[:, None]), page, table))
    i, b = _owner(kv, st["kv_indices"].numel())
    listed_page = table[b, (i - kv[b]).clamp(0, table.shape[1] - 1)]
    st["kv_indices"].copy_(torch.where(i < kv[-1], listed_page, st["kv_indices"]))
    i, b = _owner(qo, st["positions"].numel())
    position = held[b] - new[b] + i - qo[b]
    page = table[b, (position // ps).clamp(0, table.shape[1] - 1)].long()
    live = i < qo[-1]
    return dict(qo_indptr=qo.int(), key_indptr=_running(held).int(), kv_indptr=kv.int(),
                kv_indices=st["kv_indices"], block_table=table,
                kv_last_page_lens=(held - (pages - 1) * ps).clamp(min=1).int(),
                free_count=(st["free_count"] - taken[-1]).int(),
                positions=torch.where(live, position, 0).int(),
                slots=torch.where(live, page * ps + position % ps, -1).int())


def _rotate(x, cos_sin, positions, neox):
    """fp32 (tokens, heads, dim) with its first columns rotated by the table's rows."""
    r = cos_sin.shape[1]
    row = cos_sin[positions.long()][:, None, :]
    c, s = row[..., :r // 2], row[..., r // 2:]
    rot, rest = x[..., :r], x[..., r:]
    if neox:
        a, b = rot[..., :r // 2], rot[..., r // 2:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], dim=-1)
    a, b = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2), rest], dim=-1)


def _held(st):
    """Positions of every request, from its page list."""
    pages = (st["kv_indptr"][1:] - st["kv_indptr"][:-1]).long()
    return torch.where(pages > 0, (pages - 1) * st["case"]["page"] + st["kv_last_page_lens"], 0)


def _power(largest):
    """The smallest power of two s with largest <= 448 s, between 2^-60 and 2^120."""
    part, exponent = torch.frexp(largest)
    k = torch.where(largest > 0, exponent - 9 + (part > 0.875).int(), -60).clamp(-60, 120)
    return ((k.int() + 127) << 23).view(torch.float32)


def _bytes(x):
    return x.view(torch.uint8)


def _requantise(x, cache, scale, rows, fresh, old, fp8=torch.float8_e4m3fn):
    """Writes fp32 rows x (tokens, heads, dim) into one cache.  rows: (page, slot, block) of each
    token; fresh: whether its block starts in this call; old: (page, slots, block, earlier) of the
    block that each request's first token continues."""
    page, slot, block = rows
    largest = torch.zeros_like(scale).index_put_((page, block), x.new_zeros(()))
    flat = (page * scale.shape[1] + block)[:, None].expand(-1, x.shape[1])
    largest.view(-1, scale.shape[2]).scatter_reduce_(0, flat, x.abs().amax(-1), "amax")
    started = torch.zeros(scale.shape[:2], dtype=torch.bool, device=DEV)
    started[page, block] = fresh
    touched = torch.zeros_like(started)
    touched[page, block] = True
    power = _power(largest)
    after = torch.where(touched[..., None],
                        torch.where(started[..., None], power, torch.maximum(scale, power)), scale)
    o_page, o_slot, o_block, earlier = old
    ratio = (scale / after)[o_page, o_block]                      # (requests, heads)
    codes = _bytes(cache)[o_page[:, None], o_slot].view(fp8).float() * ratio[:, None, :, None]
    at = torch.nonzero(earlier, as_tuple=True)
    _bytes(cache)[o_page[at[0]], o_slot[at]] = _bytes(codes[at].to(fp8))
    coded = (x / after[page, block][..., None]).clamp(-448, 448).to(fp8)
    _bytes(cache)[page, slot] = _bytes(coded)
    scale.copy_(after)


def _plain_append(st):
    case = st["case"]
    ps, bs = case["page"], case["block"]
    q = _rotate(st["q"].float(), st["cos_sin"], st["positions"], case["neox"])
    k = _rotate(st["k"].float(), st["cos_sin"], st["positions"], case["neox"])
    qo, kv, held = st["qo_indptr"].long(), st["kv_indptr"].long(), _held(st)
    new = qo[1:] - qo[:-1]
    begin = held - new
    i, b = _owner(qo, st["q"].shape[0])
    position = begin[b] + i - qo[b]
    page = st["kv_indices"].long()[kv[b] + position // ps]
    rows = (page, position % ps, position % ps // bs)
    fresh = begin[b] <= position // bs * bs
    # the block that a request's first new token continues: its earlier slots
    some = torch.nonzero((begin % bs > 0) & (new > 0))[:, 0]
    first = begin[some]
    o_page = st["kv_indices"].long()[kv[some] + first // ps]
    o_slot = (first // bs * bs % ps)[:, None] + torch.arange(bs, device=DEV)
    old = (o_page, o_slot, first % ps // bs, torch.arange(bs, device=DEV) < (first % bs)[:, None])
    for x, name in ((k, "k"), (st["v"].float(), "v")):
        _requantise(x, st[name + "_cache"], st[name + "_scale"], rows, fresh, old)
    out = dict(q=q.bfloat16(), k_cache=st["k_cache"], v_cache=st["v_cache"], k_scale=st["k_scale"],
               v_scale=st["v_scale"])
    if st["k_out"] is not None:
        out["k"] = k.bfloat16()
    return out


def _dequantised(st, name, page, slot):
    """fp32 entries (..., heads, dim) of one cache at (page, slot)."""
    cache = st[name + "_cache"]
    scale = st[name + "_scale"][page, slot // st["case"]["block"]]
    return _bytes(cache)[page, slot].view(cache.dtype).float() * scale[..., None]


def _plain_gather(st):
    ps = st["case"]["page"]
    start, kv, qo, held = st["key_indptr"].long(), st["kv_indptr"].long(), st["qo_indptr"].long(), _held(st)
    i, b = _owner(start, st["k_rows"].shape[0])
    position = (i - start[b]).clamp(max=(held[b] - 1).clamp(min=0))
    page = st["kv_indices"].long()[(kv[b] + position // ps).clamp(max=st["kv_indices"].numel() - 1)]
    at = held[b] - (qo[b + 1] - qo[b])               # the first position that is new
    fresh = (position >= at)[:, None, None]
    token = (qo[b] + position - at).clamp(0, st["k_new"].shape[0] - 1)
    live = (i < start[-1])[:, None, None]
    rows = {}
    for name in ("k", "v"):
        cached = _dequantised(st, name, page, position % ps).bfloat16()
        x = torch.where(fresh, st[name + "_new"][token], cached)
        rows[name] = torch.where(live, x, st[name + "_rows"])
    return rows


def _plain_decode(st):
    case = st["case"]
    hk, ps, d, t = case["kv_heads"], case["page"], case["dim"], case["new"]
    group = case["q_heads"] // hk
    kv, held = st["kv_indptr"].long(), _held(st)
    n = held.numel()
    j = torch.arange(max(1, max(_lengths(case)[1])), device=DEV)
    at = (kv[:-1, None] + (j // ps)[None, :]).clamp(max=max(0, st["kv_indices"].numel() - 1))
    page = st["kv_indices"].long()[at] if st["kv_indices"].numel() else torch.zeros_like(at)
    k = _dequantised(st, "k", page, (j % ps)[None, :].expand_as(page)).permute(0, 2, 3, 1)
    q = st["q"].float().view(n, t, hk, group, d).permute(0, 2, 1, 3, 4).reshape(n, hk, t * group, d)
    s = torch.matmul(q, k).view(n, hk, t, group, -1) * st["sm_scale"]
    del k
    last = held[:, None] - t + torch.arange(t, device=DEV)              # the last position seen
    s.masked_fill_((j > last[..., None])[:, None, :, None, :], -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
    s = s.sub_(top).exp_()
    z = s.sum(dim=-1, keepdim=True)
    v = _dequantised(st, "v", page, (j % ps)[None, :].expand_as(page)).permute(0, 2, 1, 3)
    v = torch.where((j < held[:, None])[:, None, :, None], v, torch.zeros((), device=DEV))
    o = torch.matmul(s.view(n, hk, t * group, -1), v).view(n, hk, t, group, d)
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(n * t, -1, d)
    lse = (top + torch.log(z))[..., 0].permute(0, 2, 1, 3).reshape(n * t, -1)
    return dict(o=o.bfloat16(), lse=lse)


_plain = {"table": _plain_table, "append": _plain_append, "gather": _plain_gather, "decode": _plain_decode}


def _own_table(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_build_page_table(st["seq_lens"], st["new_lens"], st["block_table"], st["case"]["page"],
                            st["qo_indptr"], st["key_indptr"], st["kv_indptr"], st["kv_indices"],
                            st["kv_last_page_lens"], st["error_word"], positions=st["positions"],
                            slot_mapping=st["slots"], free_pages=st["free_pages"],
                            free_count=st["free_count"], free_count_out=st["free_count_out"])
    out = {name: st[name] for name in ("qo_indptr", "key_indptr", "kv_indptr", "kv_indices", "block_table",
                                       "kv_last_page_lens", "positions", "slots")}
    return dict(out, free_count=st["free_count_out"])


def _own_append(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_gqa_block_append(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"],
                            int(st["case"]["neox"]), st["qo_indptr"], st["kv_indptr"], st["kv_indices"],
                            st["kv_last_page_lens"], st["q_out"], st["k_cache"], st["v_cache"],
                            st["k_scale"], st["v_scale"], st["error_word"], k_out=st["k_out"])
    out = dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"], k_scale=st["k_scale"],
               v_scale=st["v_scale"])
    if st["k_out"] is not None:
        out["k"] = st["k_out"]
    return out


def _own_gather(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_gqa_block_gather(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["kv_indptr"],
                            st["kv_indices"], st["kv_last_page_lens"], st["key_indptr"], st["k_rows"],
                            st["v_rows"], st["error_word"], qo_indptr=st["qo_indptr"], k_new=st["k_new"],
                            v_new=st["v_new"])
    return dict(k=st["k_rows"], v=st["v_rows"])


def _own_decode(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_gqa_block_decode(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["o"],
                            st["qo_indptr"], st["kv_indptr"], st["kv_indices"], st["kv_last_page_lens"],
                            st["case"]["new"], st["sm_scale"], lse_out=st["lse"], workspace=st["workspace"])
    return dict(o=st["o"], lse=st["lse"])


_own = {"table": _own_table, "append": _own_append, "gather": _own_gather, "decode": _own_decode}


# ----------------------------------------------------------------------------- fp64

def exact(case, seed):
    if case["op"] == "table":
        return None                                  # whole numbers only
    st = _INPUTS[case["op"]](case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "decode": _exact_decode}[case["op"]](st)


def _slots_of(st, b, positions):
    """Cache slots (page * PS + slot) of positions of request b."""
    start = int(st["kv_indptr"][b])
    ps = st["case"]["page"]
    return st["kv_indices"][start + positions // ps].long() * ps + positions % ps


def _flat(st, name):
    """(codes, scale of each slot) of one cache in fp64, slots in one line."""
    case = st["case"]
    codes = st[name + "_cache"].double().flatten(0, 1)
    return codes, st[name + "_scale"].double().repeat_interleave(case["block"], dim=1).flatten(0, 1)


def _exact_append(st):
    """Each pair as a complex number, turned by the table's unit (cos + i sin); block by block."""
    case = st["case"]
    r, bs, hk = case["rot"], case["block"], case["kv_heads"]
    row = st["cos_sin"].double()[st["positions"].long()]
    turn = torch.complex(row[:, :r // 2], row[:, r // 2:])[:, None, :]
    first = torch.arange(r // 2, device=DEV) * (1 if case["neox"] else 2)
    second = first + (r // 2 if case["neox"] else 1)
    turned = []
    for x in (st["q"], st["k"]):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first] = z.real
        y[..., second] = z.imag
        turned.append(y)
    out = dict(q=turned[0])
    new, held = _lengths(case)
    for name, x in (("k", turned[1]), ("v", st["v"].double())):
        codes, scale = _flat(st, name)
        block_scale = st[name + "_scale"].double().flatten(0, 1)
        at = 0
        for b, (t, n) in enumerate(zip(new, held)):
            if t == 0:
                continue
            begin = n - t
            low, high = begin // bs * bs, -(-n // bs) * bs
            padded = torch.zeros(high - low, hk, case["dim"], dtype=torch.float64, device=DEV)
            padded[begin - low:n - low] = x[at:at + t]
            top = padded.view(-1, bs, hk, case["dim"]).abs().amax(dim=(1, 3))
            part, exponent = torch.frexp(top / 448)  # part in [0.5, 1), 0.5 for powers of two
            exponent = torch.where(part > 0.5, exponent, exponent - 1)
            power = torch.exp2(torch.where(top > 0, exponent, -60).clamp(-60, 120).double())
            where = _slots_of(st, b, torch.arange(low, n, device=DEV))
            blocks = where[::bs] // bs
            if begin > low:                          # the first block holds earlier tokens
                before = block_scale[blocks[0]]
                power[0] = torch.maximum(power[0], before)
                codes[where[:begin - low]] *= (before / power[0])[None, :, None]
            block_scale[blocks] = power
            per_row = power.repeat_interleave(bs, dim=0)[begin - low:n - low]
            codes[where[begin - low:]] = (x[at:at + t] / per_row[..., None]).clamp(-448, 448)
            at += t
        out[name + "_cache"] = codes.view(st[name + "_cache"].shape)
        out[name + "_scale"] = block_scale.view(st[name + "_scale"].shape)
    if st["k_out"] is not None:
        out["k"] = turned[1]
    return out


def _exact_gather(st):
    new, held = _lengths(st["case"])
    out = {}
    for name in ("k", "v"):
        codes, scale = _flat(st, name)
        rows = st[name + "_rows"].double()
        at = token = 0
        for b, (t, n) in enumerate(zip(new, held)):
            if n > t:
                where = _slots_of(st, b, torch.arange(n - t, device=DEV))
                rows[at:at + n - t] = codes[where] * scale[where][..., None]
            rows[at + n - t:at + n] = st[name + "_new"][token:token + t].double()
            at, token = at + n, token + t
        out[name] = rows
    return out


def _exact_decode(st):
    """One request and one KV head at a time; softmax through the log of the sum."""
    case = st["case"]
    hk, t, bs = case["kv_heads"], case["new"], case["block"]
    group = case["q_heads"] // hk
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(case)[1]):
        if n == 0:
            continue
        where = _slots_of(st, b, torch.arange(n, device=DEV))
        tokens = slice(b * t, (b + 1) * t)
        seen = torch.arange(n, device=DEV)[None, :] <= n - t + torch.arange(t, device=DEV)[:, None]
        some = seen.any(dim=1)
        seen = seen.repeat_interleave(group, dim=0)
        for h in range(hk):
            one = {}
            for name in ("k", "v"):
                codes = _bytes(st[name + "_cache"]).flatten(0, 1)[:, h].index_select(0, where).view(torch.float8_e4m3fn)
                scale = st[name + "_scale"].flatten(0, 1)[:, h].index_select(0, where // bs)
                one[name] = codes.double() * scale.double()[:, None]
            heads = slice(h * group, (h + 1) * group)
            q = st["q"][tokens, heads].double().reshape(t * group, -1)
            s = torch.where(seen, torch.einsum("rd,nd->rn", q, one["k"]) * st["sm_scale"], -math.inf)
            l = torch.logsumexp(s, dim=1)
            p = torch.where(seen, torch.exp(s - l.clamp(min=-1e300)[:, None]), 0.0)
            lse[tokens, heads] = torch.where(some[:, None], l.view(t, group), -math.inf)
            o[tokens, heads] = torch.einsum("rn,nd->rd", p, one["v"]).view(t, group, -1)
    return dict(o=o, lse=lse)

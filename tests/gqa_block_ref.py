"""Plain restatements of the operators over caches with a scale for each block and head, request
by request and block by block, and the inputs their tests share.  Test infrastructure only."""
import math
import random

import torch

from tests import gqa_ref as ref

F8 = torch.float8_e4m3fn


def gen(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def sums(counts, device):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


def table(max_pos, r, device):
    ang = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(r // 2, device=device, dtype=torch.float64) * 2 / r)
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


# ------------------------------------------------------------------------- page tables

def page_table(seq, new, rows, ps, free=None, n_idx=None):
    """The lists of a step as whole numbers.  rows: the block table as lists (changed in place);
    free: the stack of free pages, bottom first (changed in place).  Returns a dict of lists."""
    out = dict(qo=[0], key=[0], kv=[0], idx=[], last=[], pos=[], slots=[])
    for b, (n, t) in enumerate(zip(seq, new)):
        if n < 0 or t < 0 or t > n or -(-n // ps) > len(rows[b]):
            n = t = 0
        pages, had = -(-n // ps), -(-(n - t) // ps)
        if free is not None:
            for j in range(had, pages):
                rows[b][j] = free.pop() if free else -1
        out["idx"] += rows[b][:pages]
        out["kv"].append(out["kv"][-1] + pages)
        out["qo"].append(out["qo"][-1] + t)
        out["key"].append(out["key"][-1] + n)
        out["last"].append(n - (pages - 1) * ps)
        for p in range(n - t, n):
            page = rows[b][p // ps]
            out["pos"].append(p)
            out["slots"].append(page * ps + p % ps if page >= 0 else -1)
    return out


# ------------------------------------------------------------------------------ caches

def caches(pages, ps, bs, hk, d, layout, device):
    """Empty caches (codes 0x7F, which is NaN; scales NaN): slots outside heads ("nhd"), heads
    outside slots ("hnd"), or keys and values in one tensor of wider rows ("shared"), scales with
    their dims in another order."""
    if layout == "shared":
        both = torch.zeros(pages, 2, ps, hk, d + 16, dtype=torch.uint8, device=device)
        k, v = both[:, 0, :, :, :d], both[:, 1, :, :, :d]
    elif layout == "hnd":
        k, v = (torch.zeros(pages, hk, ps, d, dtype=torch.uint8, device=device).transpose(1, 2) for _ in range(2))
    else:
        k, v = (torch.zeros(pages, ps, hk, d, dtype=torch.uint8, device=device) for _ in range(2))
    nb = ps // bs
    if layout == "nhd":
        ks, vs = (torch.zeros(pages, nb, hk, device=device) for _ in range(2))
    elif layout == "hnd":
        ks, vs = (torch.zeros(hk, pages, nb, device=device).permute(1, 2, 0) for _ in range(2))
    else:
        wide = torch.zeros(pages, hk, nb, 3, device=device)
        ks, vs = wide[..., 0].transpose(1, 2), wide[..., 2].transpose(1, 2)
    for t in (k, v):
        t.fill_(0x7F)
    for t in (ks, vs):
        t.fill_(math.nan)
    return k.view(F8), v.view(F8), ks, vs


def put(cache, where, codes):
    """cache[page, slot] = codes for where = (pages, slots)."""
    cache.view(torch.uint8)[where] = codes.view(torch.uint8)


def take(cache, where):
    return cache.view(torch.uint8)[where].view(F8)


class Pages:
    """Page lists of requests with `held` positions over shuffled pages of a pool."""

    def __init__(self, held, ps, bs, device, seed=0, spare=3):
        self.held, self.ps, self.bs, self.device = held, ps, bs, device
        counts = [-(-n // ps) for n in held]
        self.pool = sum(counts) + spare
        ids = list(range(self.pool))
        random.Random(seed).shuffle(ids)
        self.lists, at = [], 0
        for n in counts:
            self.lists.append(ids[at:at + n])
            at += n
        self.indptr = sums(counts, device)
        tail = [1 << 30] * 5                                  # never read
        self.indices = torch.tensor(ids[:at] + tail, dtype=torch.int32, device=device)
        self.last = torch.tensor([n - (c - 1) * ps if n else 1 for n, c in zip(held, counts)],
                                 dtype=torch.int32, device=device)

    def where(self, b, lo, hi):
        """(pages, slots) of positions [lo, hi) of request b."""
        p = torch.arange(lo, hi, device=self.device)
        ids = torch.tensor(self.lists[b] or [0], device=self.device)
        return ids[p // self.ps], p % self.ps

    def block(self, b, at):
        """(page, block) of position `at` of request b."""
        return self.lists[b][at // self.ps], at % self.ps // self.bs


def fill(pages, cache, scale, g, lens=None, exponents=(-9, -4), std=100.0):
    """Random codes and power-of-two scales at the first lens[b] positions of every request (slots
    behind stay poison, scales of blocks without a position stay NaN)."""
    hk, d = cache.shape[2:]
    for b, n in enumerate(pages.held if lens is None else lens):
        if n == 0:
            continue
        x = (torch.randn(n, hk, d, generator=g, device=pages.device) * std).clamp(-448, 448).to(F8)
        put(cache, pages.where(b, 0, n), x)
        for at in range(0, n, pages.bs):
            e = torch.randint(*exponents, (hk,), generator=g, device=pages.device).float()
            scale[pages.block(b, at)] = torch.exp2(e)


# ------------------------------------------------------------------------------ append

def turned(x, cos_sin, positions, neox):
    """fp32, every operation rounded on its own (torch's elementwise operations round so)."""
    r = cos_sin.shape[1]
    row = cos_sin[positions.long()][:, None]
    c, s = row[..., :r // 2], row[..., r // 2:]
    x = x.float()
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if neox else (x[..., 0:r:2], x[..., 1:r:2])
    u, w = a * c - b * s, b * c + a * s
    front = torch.cat([u, w], -1) if neox else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([front, x[..., r:]], -1)


def fit(a):
    """The smallest power of two s with a <= 448 s, from 2^-60 to 2^120, by trying them (fp64)."""
    k = -60
    while k < 120 and a > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def coded(x, scale):
    return (x / scale).clamp(-448, 448).to(F8)


def append(pages, new, rows, cache, scale):
    """Writes fp32 rows (T, Hk, D) behind the cached positions, block by block and head by head."""
    at, hk = 0, rows.shape[1]
    for b, (t, n) in enumerate(zip(new, pages.held)):
        begin = n - t
        for first in range(begin // pages.bs * pages.bs, n, pages.bs) if t else ():
            lo, hi = max(first, begin), min(first + pages.bs, n)
            x = rows[at + lo - begin:at + hi - begin]
            for h in range(hk):
                y = x[:, h]
                a = torch.where(y.isfinite(), y.abs(), 0.0).max().item()
                s = fit(a)
                blk = (*pages.block(b, first), h)
                if lo > first:
                    old = scale[blk].clone()
                    if s > old.item():
                        w = pages.where(b, first, lo)
                        codes = take(cache, w)[:, h].float() * (old / torch.tensor(s, device=old.device))
                        kept = take(cache, w)
                        kept.view(torch.uint8)[:, h] = codes.clamp(-448, 448).to(F8).view(torch.uint8)
                        put(cache, w, kept)
                    else:
                        s = old.item()
                scale[blk] = s
                w = pages.where(b, lo, hi)
                kept = take(cache, w)
                kept.view(torch.uint8)[:, h] = coded(y, scale[blk]).view(torch.uint8)
                put(cache, w, kept)
        at += t


# ---------------------------------------------------------------------- gather, decode

def values(pages, b, cache, scale, n=None):
    """fp32 (n, Hk, D): codes times scales of request b's first n positions."""
    n = pages.held[b] if n is None else n
    page, slot = pages.where(b, 0, n)
    return take(cache, (page, slot)).float() * scale[page, slot // pages.bs][..., None]


# A weight (with its v scale) is rounded to f16 where the largest counts 2^14; below f16's normal
# range it loses half of 2^-24, 2^-39 of the largest.
WEIGHT = ref.F16
LOST = 2.0 ** -39
# With more than 16 rows a KV head the rounded weight counts at least 2^5 where it is largest and is
# written as three e4m3 codes h + 2^-5 l + 2^-10 l', exact down to the last one's smallest step,
# 2^-9 2^-10: half of it is 2^-25 of the largest.
LOST_MANY = 2.0 ** -25


def attend(pages, b, q, k_cache, v_cache, ks, vs, sm, least=LOST):
    """o, lse, mass and largest score of the newest q.shape[0] tokens of request b, fp64, and what
    their smallest weights can lose."""
    t, hq, d = q.shape
    hk = k_cache.shape[2]
    group, n = hq // hk, pages.held[b]
    k, v = values(pages, b, k_cache, ks).double(), values(pages, b, v_cache, vs).double()
    page, slot = pages.where(b, 0, n)
    scale = vs[page, slot // pages.bs].double().clamp_min(2.0 ** -60)       # (n, hk)
    codes = take(v_cache, (page, slot)).float().double().abs().sum(0)       # (hk, d)
    limit = (n - t + 1 + torch.arange(t, device=q.device)).repeat_interleave(group)
    out = []
    for h in range(hk):
        qq = q[:, h * group:(h + 1) * group].double().reshape(t * group, d)
        o, lse, mass, big = ref.attend(qq, k[:, h], v[:, h], sm, limit)
        if n:
            s = torch.where(torch.arange(n, device=q.device) < limit[:, None], qq @ k[:, h].T * sm, -math.inf)
            w = torch.exp(s - lse.clamp_min(-1e300)[:, None]) * scale[:, h]
            lost = least * w.amax(1, keepdim=True) * codes[h]
        else:
            lost = torch.zeros_like(o)
        out.append((o, lse, mass, big, lost))
    back = lambda x: x.view(t, group, *x.shape[1:])
    return [torch.cat([back(x) for x in y], dim=1) for y in zip(*out)]


def check(got_o, got_lse, want, n_keys, d, out_eps, what):
    """As ref.check, with what the smallest weights lose."""
    o, lse, mass, big, lost = want
    empty = torch.isneginf(lse)
    ob, lb = ref.bounds(o, torch.where(empty, torch.zeros_like(lse), lse), mass, big, n_keys, d, WEIGHT, out_eps)
    g = got_o.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    worst = ((g - o).abs() / (ob + lost)).max().item()
    assert worst <= 1.0, f"{what}: o error {worst:.3f} of its bound"
    assert (g[empty] == 0).all(), f"{what}: an empty row is not zero"
    gl = got_lse.double()
    assert torch.equal(torch.isneginf(gl), empty), f"{what}: lse of empty rows"
    worst = (torch.where(empty, torch.zeros_like(gl), (gl - lse).abs()) / lb).max().item()
    assert worst <= 1.0, f"{what}: lse error {worst:.3f} of its bound"

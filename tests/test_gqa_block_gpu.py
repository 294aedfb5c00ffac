"""The append, the gather and the attention over caches with a scale for each block and head."""
import math

import pytest
import torch

from tests import gqa_block_ref as blk
from tests import gqa_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).bfloat16()


def _same(a, b):
    """Equal bits, any NaN equal to any other."""
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    af, bf = a.float().isnan(), b.float().isnan()
    return torch.equal(af, bf) and torch.equal(a.view(kind)[~af], b.view(kind)[~bf])


# -------------------------------------------------------------------------------- append

class Append:
    def __init__(self, new, before, Hq, Hk, D, R, neox, ps, bs, layout="nhd", seed=0, pad=0):
        self.g = blk.gen(seed + sum(new) + D + bs, DEV)
        self.new, self.neox = new, neox
        held = [t + c for t, c in zip(new, before)]
        self.pages = blk.Pages(held, ps, bs, DEV, seed)
        self.kc, self.vc, self.ks, self.vs = blk.caches(self.pages.pool, ps, bs, Hk, D, layout, DEV)
        blk.fill(self.pages, self.kc, self.ks, self.g, before, (-14, -6))
        blk.fill(self.pages, self.vc, self.vs, self.g, before, (-14, -6))
        T = sum(new) + pad
        # q, k and v as views of one projection, rows of different sizes
        spread = torch.exp2(torch.randn(T, 1, generator=self.g, device=DEV) * 2)
        qkv = (torch.randn(T, (Hq + 2 * Hk) * D + 8, generator=self.g, device=DEV) * spread).bfloat16()
        self.q = qkv[:, :Hq * D].view(T, Hq, D)
        self.k = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        self.v = qkv[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(T, Hk, D)
        self.qo = blk.sums(new, DEV)
        self.pos = torch.randint(0, 500, (T,), generator=self.g, device=DEV, dtype=torch.int32)
        self.cs = blk.table(500, R, DEV)
        self.q_out = torch.full((T, Hq, D + 8), math.nan, dtype=torch.bfloat16, device=DEV)[:, :, :D]
        self.k_out = torch.full((T, Hk, D), math.nan, dtype=torch.bfloat16, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, pm, q_out=None, k_out=None, **kw):
        pm.mla_gqa_block_append(self.q, self.k, self.v, self.pos, self.cs, self.neox, self.qo,
                                self.pages.indptr, self.pages.indices, self.pages.last,
                                self.q_out if q_out is None else q_out, self.kc, self.vc, self.ks, self.vs,
                                self.err, k_out=self.k_out if k_out is None else k_out, **kw)

    def copies(self):
        return [x.clone() for x in (self.kc.view(torch.uint8), self.vc.view(torch.uint8), self.ks, self.vs)]

    def want(self):
        """What the definition leaves: the caches and scales after, and the rotated rows."""
        kc, vc, ks, vs = self.copies()
        kc, vc = kc.view(blk.F8), vc.view(blk.F8)
        n = sum(self.new)
        q, k = (blk.turned(x[:n], self.cs, self.pos[:n], self.neox) for x in (self.q, self.k))
        blk.append(self.pages, self.new, k, kc, ks)
        blk.append(self.pages, self.new, self.v[:n].float(), vc, vs)
        return kc, vc, ks, vs, q.bfloat16(), k.bfloat16()

    def check(self, want):
        kc, vc, ks, vs, q, k = want
        n = sum(self.new)
        assert _same(self.ks, ks), "scales of keys"
        assert _same(self.vs, vs), "scales of values"
        assert _same(self.kc, kc), "codes of keys"
        assert _same(self.vc, vc), "codes of values"
        assert _same(self.q_out[:n], q) and _same(self.k_out[:n], k)
        assert self.q_out[n:].isnan().all() and self.k_out[n:].isnan().all()


APPENDS = [
    # new, before, Hq, Hk, D, R, neox, ps, bs, layout
    ([1], [0], 1, 1, 64, 16, 1, 1, 1, "nhd"),
    ([1], [0], 8, 2, 128, 128, 1, 16, 16, "nhd"),
    ([1, 1, 1, 1], [5, 16, 15, 130], 8, 2, 128, 128, 0, 16, 16, "hnd"),
    ([1] * 9, [0, 1, 127, 128, 129, 255, 63, 64, 300], 16, 2, 128, 64, 1, 128, 128, "nhd"),
    ([1] * 9, [0, 1, 127, 128, 129, 255, 63, 64, 300], 5, 5, 64, 64, 0, 128, 64, "shared"),
    ([0, 3, 0, 0, 40, 0], [7, 2, 0, 33, 100, 0], 6, 2, 64, 32, 1, 4, 4, "hnd"),
    ([0, 3, 0, 0, 40, 0], [7, 2, 0, 33, 100, 0], 6, 2, 128, 32, 0, 8, 2, "nhd"),
    ([17, 1, 130], [3, 0, 50], 9, 1, 128, 96, 1, 32, 8, "shared"),
    ([17, 1, 130], [3, 0, 50], 9, 1, 64, 48, 0, 32, 8, "shared"),
    ([300], [0], 4, 4, 128, 128, 0, 1024, 128, "nhd"),
    ([300], [77], 3, 3, 64, 16, 1, 512, 128, "hnd"),
    ([257, 31, 64], [1, 90, 64], 25, 5, 64, 32, 0, 64, 32, "nhd"),
    ([100, 200, 150], [31, 32, 33], 14, 2, 128, 80, 1, 64, 64, "hnd"),
    ([33, 20], [0, 6], 7, 7, 128, 128, 1, 1, 1, "nhd"),
    ([33, 20], [1, 6], 16, 1, 64, 64, 1, 2, 1, "hnd"),
    ([128, 256], [128, 384], 8, 8, 64, 64, 0, 128, 128, "nhd"),
    ([5] * 40, [i * 7 % 140 for i in range(40)], 4, 2, 128, 128, 1, 128, 128, "nhd"),
    ([20] * 40, [i * 7 % 140 for i in range(40)], 2, 2, 128, 128, 0, 128, 128, "hnd"),
    # more than two waves of keys' and values' blocks, with the queries' between them
    ([1000], [5], 256, 64, 128, 128, 1, 16, 16, "nhd"),
    ([1900], [5], 256, 64, 64, 32, 0, 64, 32, "hnd"),
]


@pytest.mark.parametrize("case", APPENDS)
def test_append_is_exact(pm, case):
    a = Append(*case)
    want = a.want()
    a.run(pm)
    assert a.err.item() == 0
    a.check(want)


@pytest.mark.parametrize("bs", [1, 16, 128])
def test_append_many_requests(pm, bs):
    """More requests than one probe of 31 finds, idle ones between; behind them a padded batch."""
    new = [(i * 5) % 3 for i in range(1100)]
    a = Append(new, [(i * 11) % 40 for i in range(1100)], 2, 1, 64, 64, 1, 128 if bs > 1 else 8, bs, pad=29)
    want = a.want()
    a.run(pm)
    assert a.err.item() == 0
    a.check(want)


@pytest.mark.parametrize("neox", [0, 1])
@pytest.mark.parametrize("new,bs", [([40, 1, 200], 128), ([1, 1, 30, 1, 1, 1, 1, 1, 1], 128), ([40, 3], 16)])
def test_append_in_place(pm, neox, new, bs):
    a, b = (Append(new, [9] * len(new), 6, 2, 64, 64, neox, 128, bs) for _ in range(2))
    want = a.want()
    a.run(pm, q_out=a.q, k_out=a.k)
    n = sum(new)
    assert _same(a.q[:n], want[4]) and _same(a.k[:n], want[5])
    a.q_out, a.k_out = a.q, a.k
    a.check(want)
    b.run(pm)
    assert torch.equal(a.kc.view(torch.uint8), b.kc.view(torch.uint8))


def test_append_twice_is_the_same(pm):
    """The same step once more over its own slots: nothing moves (a block's scale does not grow
    for values that it holds)."""
    a = Append([30, 1, 200], [9, 100, 250], 4, 2, 128, 128, 1, 128, 64)
    a.run(pm)
    once = a.copies()
    a.run(pm)
    for x, y in zip(once, a.copies()):
        assert _same(x, y)


@pytest.mark.parametrize("D", [64, 128])
def test_append_token_by_token(pm, D):
    """A request appended one token a call.  Against all at once: the same scales in the end, and
    codes that passed through grown scales off by what e4m3's subnormals lose each time: half of
    2^-9 of the scale a growth, summed over at most all growths below half a step of the last."""
    n, bs, Hk = 50, 16, 2
    whole = Append([n], [0], 4, Hk, D, D, 1, 16, bs)
    whole.run(pm)
    step = Append([n], [0], 4, Hk, D, D, 1, 16, bs)
    for i in range(n):
        step.pages.held[0] = i + 1
        one = torch.tensor([0, i // 16 + 1], dtype=torch.int32, device=DEV)
        last = torch.tensor([i % 16 + 1], dtype=torch.int32, device=DEV)
        pm.mla_gqa_block_append(step.q[i:i + 1], step.k[i:i + 1], step.v[i:i + 1], step.pos[i:i + 1], step.cs, 1,
                                torch.tensor([0, 1], dtype=torch.int32, device=DEV), one, step.pages.indices,
                                last, step.q_out[i:i + 1], step.kc, step.vc, step.ks, step.vs, step.err)
    assert step.err.item() == 0
    assert _same(step.ks, whole.ks) and _same(step.vs, whole.vs)
    for c in ("k", "v"):
        x, y = (blk.values(a.pages, 0, getattr(a, c + "c"), getattr(a, c + "s"), n) for a in (step, whole))
        last = getattr(whole, c + "s")
        page, slot = whole.pages.where(0, 0, n)
        unit = last[page, slot // bs][..., None] * 2.0 ** -9
        # growths by 2, 4, ...: the losses form a geometric sum below one subnormal step; the once
        # rounded value then differs by at most a further half step
        assert ((x - y).abs() <= 1.5 * unit).all()
        # normal codes are the same bits
        normal = y.abs() >= unit * 2 ** 4
        assert torch.equal(x[normal], y[normal])


def test_append_infinities_nan_and_zeros(pm):
    a = Append([20, 3, 1], [0, 16, 8], 1, 1, 64, 16, 1, 16, 16)
    v = a.v.clone()
    v[0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 3e38, -3e38, 1e-38], device=DEV).bfloat16()
    v[16:20] = 0                      # a block of zeros
    v[20:23] = math.nan               # a block of nothing finite
    v[23] = math.inf                  # joins a block that has a scale
    a.v = v
    k = a.k.clone()
    k[17, 0, 40] = math.inf           # a column that passes through
    a.k = k
    want = a.want()
    a.run(pm)
    assert a.err.item() == 0
    a.check(want)
    assert a.vs[a.pages.block(0, 16)].item() == 2.0 ** -60
    assert a.vs[a.pages.block(1, 16)].item() == 2.0 ** -60


@pytest.mark.parametrize("old", [0.0237, 1e-3, 2.0 ** 61, 0.0, 3e-13, 5e30])
def test_append_continues_any_scale(pm, old):
    """Scales that someone else wrote: no power of two, zero, tiny, huge."""
    a = Append([3, 40, 1], [5, 100, 31], 2, 2, 128, 128, 0, 128, 32)
    for s in (a.ks, a.vs):
        s.copy_(torch.where(s.isnan(), s, torch.full_like(s, old)))
    want = a.want()
    a.run(pm)
    a.check(want)


def test_append_device_errors(pm):
    """Bad pages, positions and lists: flagged, the others' entries land, nothing else is written."""
    case = ([4, 20, 2], [0, 3, 40], 2, 1, 64, 32, 1, 16, 16)
    a, b = Append(*case), Append(*case)
    want = a.want()
    bad = a.pages.indices.clone()
    bad[1] = a.pages.pool             # request 1's first page
    a.pages.indices, good = bad, a.pages.indices
    a.run(pm)
    assert a.err.item() == 64
    assert _same(a.q_out, want[4]) and _same(a.k_out, want[5])
    untouched = a.pages.where(1, 0, 16)
    for got, ref_, before in ((a.kc, want[0], b.kc), (a.vc, want[1], b.vc)):
        mine, expected = got.view(torch.uint8).clone(), ref_.view(torch.uint8).clone()
        assert torch.equal(mine[untouched], before.view(torch.uint8)[untouched])
        mine[untouched] = expected[untouched]
        assert torch.equal(mine, expected)
    # a position outside the table
    a = Append(*case)
    want = a.want()
    a.pos[5] = 500
    a.run(pm)
    assert a.err.item() == 1
    assert a.q_out[5, :, :32].isnan().all() and a.k_out[5, :, :32].isnan().all()
    assert not a.q_out[5, :, 32:].isnan().any()
    page, slot = (x[1].item() for x in a.pages.where(1, 3, 23))
    assert a.kc[page, slot, :, :32].float().isnan().all() and not a.kc[page, slot, :, 32:].float().isnan().any()
    assert _same(a.vc, want[1])
    # lists that make no sense: that request appends nothing
    whole = Append(*case).want()[0]
    for change, lost in (("tokens", (1, 2)), ("pages", (1, 2)), ("short", (2,))):
        a, before = Append(*case), Append(*case).kc
        if change == "tokens":
            a.qo[2] = 27              # past the 26 tokens; the next starts behind its end
        elif change == "pages":
            a.pages.indptr[2] = 1 << 20
        else:
            a.pages.indptr[3] = a.pages.indptr[2].clone()     # no page for two tokens
        a.run(pm)
        assert a.err.item() == 2
        for b, n in enumerate(a.pages.held):
            w = a.pages.where(b, 0, n)
            assert _same(blk.take(a.kc, w), blk.take(before if b in lost else whole, w)), (change, b)


# -------------------------------------------------------------------------------- gather

@pytest.mark.parametrize("new,before,Hk,D,ps,bs,layout", [
    ([1], [0], 1, 64, 1, 1, "nhd"),
    ([0], [1], 2, 128, 16, 16, "hnd"),
    ([3, 0, 40, 0, 0, 17], [5, 130, 0, 0, 64, 16], 2, 64, 16, 4, "shared"),
    ([130, 1], [700, 33], 5, 128, 64, 64, "hnd"),
    ([7] * 50, [i * 13 % 90 for i in range(50)], 8, 128, 128, 128, "nhd"),
    ([1], [1500], 3, 64, 1024, 128, "nhd"),
    ([20], [40], 40, 128, 2, 1, "nhd"),       # a row of more columns than a block has threads
])
def test_gather(pm, new, before, Hk, D, ps, bs, layout):
    g = blk.gen(sum(before) + D, DEV)
    held = [a + b for a, b in zip(new, before)]
    pages = blk.Pages(held, ps, bs, DEV)
    kc, vc, ks, vs = blk.caches(pages.pool, ps, bs, Hk, D, layout, DEV)
    blk.fill(pages, kc, ks, g, before)        # the new positions' slots stay poison: never read
    blk.fill(pages, vc, vs, g, before)
    ks *= 1.37                                # no power of two: two roundings
    both = _randn(g, sum(new), 2 * Hk * D)
    k_new, v_new = both[:, :Hk * D].view(-1, Hk, D), both[:, Hk * D:].view(-1, Hk, D)
    rows = blk.sums(held, DEV)
    out = torch.full((sum(held) + 2, 2, Hk, D), 7.0, dtype=torch.bfloat16, device=DEV)
    k_rows, v_rows = out[:, 0], out[:, 1]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pm.mla_gqa_block_gather(kc, vc, ks, vs, pages.indptr, pages.indices, pages.last, rows, k_rows, v_rows,
                            err, qo_indptr=blk.sums(new, DEV), k_new=k_new, v_new=v_new)
    assert err.item() == 0
    for got, cache, scale, fresh in ((k_rows, kc, ks, k_new), (v_rows, vc, vs, v_new)):
        want, at = [], 0
        for b, t in enumerate(new):
            want += [blk.values(pages, b, cache, scale, before[b]).bfloat16(), fresh[at:at + t]]
            at += t
        assert _same(got[:sum(held)], torch.cat(want))
        assert (got[sum(held):] == 7).all()
    # every position from the cache
    blk.fill(pages, kc, ks, g)
    blk.fill(pages, vc, vs, g)
    pm.mla_gqa_block_gather(kc, vc, ks, vs, pages.indptr, pages.indices, pages.last, rows, k_rows, v_rows, err)
    assert err.item() == 0
    want = torch.cat([blk.values(pages, b, kc, ks) for b in range(len(new))]).bfloat16()
    assert _same(k_rows[:sum(held)], want)


def test_gather_many_requests_and_errors(pm):
    """More requests than fit shared memory; then lists and pages that make no sense."""
    held = [(i * 7) % 5 for i in range(1500)]
    g = blk.gen(1, DEV)
    pages = blk.Pages(held, 2, 2, DEV)
    kc, vc, ks, vs = blk.caches(pages.pool, 2, 2, 2, 64, "nhd", DEV)
    blk.fill(pages, kc, ks, g)
    blk.fill(pages, vc, vs, g)
    rows = blk.sums(held, DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k_rows, v_rows = (torch.full((sum(held), 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    call = lambda indices=pages.indices, last=pages.last: pm.mla_gqa_block_gather(
        kc, vc, ks, vs, pages.indptr, indices, last, rows, k_rows, v_rows, err)
    call()
    want = torch.cat([blk.values(pages, b, kc, ks) for b in range(len(held))]).bfloat16()
    assert err.item() == 0 and _same(k_rows, want)
    bad = pages.indices.clone()
    bad[3] = -1
    bad[4] = pages.pool
    call(indices=bad)
    assert err.item() == 64
    # the rows of list entries 3 and 4 are zeros, the others as before
    lost = torch.zeros(sum(held), dtype=torch.bool, device=DEV)
    at = page = 0
    for n in held:
        for j in range(n):
            lost[at + j] = page + j // 2 in (3, 4)
        at, page = at + n, page + -(-n // 2)
    assert lost.any() and (k_rows[lost] == 0).all() and _same(k_rows[~lost], want[~lost])
    # a request whose row range is not as long as its list
    err.zero_()
    k_rows.fill_(7.0)
    last = pages.last.clone()
    last[2] = 3 - last[2]             # request 2: one position more or less
    call(last=last)
    assert err.item() == 2
    lo, hi = rows[2].item(), rows[3].item()
    assert (k_rows[lo:hi] == 7).all() and _same(k_rows[hi:], want[hi:]) and _same(k_rows[:lo], want[:lo])
    # rows for all but part of the last request: it is left out whole
    err.zero_()
    short = torch.full((sum(held) - 1, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    end = max(i for i, n in enumerate(held) if n > 1)
    stop = sum(held[:end])
    rows, keep = rows.clone(), rows
    pages_end = pages.indptr.clone()
    rows[end + 1:] = stop + held[end]           # nothing behind it
    pages_end[end + 2:] = pages_end[end + 1]
    pm.mla_gqa_block_gather(kc, vc, ks, vs, pages_end, pages.indices, pages.last, rows, short[:stop + 1],
                            torch.empty_like(short[:stop + 1]), err)
    assert err.item() == 2 and (short[stop] == 7).all() and _same(short[:stop], want[:stop])


# -------------------------------------------------------------------------------- decode

class Decode:
    def __init__(self, held, new, Hq, Hk, D, ps, bs, layout="nhd", seed=0, std=1.5, pad=0):
        g = blk.gen(seed + sum(held) + 17 * D + ps, DEV)
        self.new = new
        self.pages = blk.Pages(held, ps, bs, DEV, seed)
        self.kc, self.vc, self.ks, self.vs = blk.caches(self.pages.pool, ps, bs, Hk, D, layout, DEV)
        blk.fill(self.pages, self.kc, self.ks, g)
        blk.fill(self.pages, self.vc, self.vs, g)
        self.q = _randn(g, sum(new) + pad, Hq, D, std=std)
        self.qo = blk.sums(new, DEV)
        self.sm = D ** -0.5

    def run(self, pm, o_dtype=torch.bfloat16, ws=None, **kw):
        o = torch.full(self.q.shape, math.nan, dtype=o_dtype, device=DEV)
        lse = torch.full(self.q.shape[:2], math.nan, device=DEV)
        ws = pm.mla_gqa_block_decode(self.q, self.kc, self.vc, self.ks, self.vs, o, self.qo, self.pages.indptr,
                                     self.pages.indices, self.pages.last, max(1, *self.new, 0), self.sm,
                                     lse, ws, **kw)
        return o, lse, ws

    def check(self, o, lse, what="", least=blk.LOST):
        at = 0
        for b, t in enumerate(self.new):
            if t == 0:
                continue
            want = blk.attend(self.pages, b, self.q[at:at + t], self.kc, self.vc, self.ks, self.vs, self.sm,
                              least)
            blk.check(o[at:at + t], lse[at:at + t], want, self.pages.held[b], self.q.shape[2],
                      ref.F32 if o.dtype == torch.float32 else ref.BF16,
                      f"{what}, request {b}: {t} of {self.pages.held[b]}")
            at += t
        assert o[at:].isnan().all() and lse[at:].isnan().all()


DECODES = [
    # held, new, Hq, Hk, D, ps, bs, layout
    ([1], [1], 1, 1, 64, 1, 1, "nhd"),
    ([1, 2, 15, 16, 17, 31, 33, 63, 64, 65], [1] * 10, 8, 2, 128, 16, 16, "nhd"),
    ([0, 5, 0, 0, 130, 0], [1, 1, 0, 1, 1, 1], 6, 2, 64, 4, 2, "hnd"),
    ([0, 0], [1, 1], 4, 2, 128, 16, 16, "nhd"),
    ([300, 7, 129], [1] * 3, 9, 1, 128, 2, 1, "shared"),
    ([2049, 1023], [1] * 2, 16, 1, 64, 1024, 128, "nhd"),
    ([511, 40, 1], [1] * 3, 33, 1, 128, 32, 8, "hnd"),
    ([257, 700], [1] * 2, 80, 2, 64, 64, 64, "nhd"),
    ([777], [1], 32, 2, 128, 128, 32, "shared"),
    ([9001, 1, 4000], [1] * 3, 5, 5, 128, 1, 1, "nhd"),
    ([20011], [1], 64, 8, 128, 128, 128, "nhd"),
    # several new tokens
    ([4], [4], 1, 1, 64, 4, 4, "nhd"),
    ([5, 40, 33, 2, 700], [4, 4, 4, 2, 3], 16, 2, 128, 16, 16, "nhd"),
    ([5, 40, 33, 2, 700], [4, 4, 4, 2, 3], 16, 2, 64, 16, 8, "hnd"),
    ([1, 2, 0, 9, 64], [4, 3, 2, 0, 5], 10, 5, 128, 8, 8, "shared"),      # queries that see nothing
    ([130, 200, 65], [64, 1, 30], 4, 4, 64, 32, 32, "nhd"),
    ([130, 200, 65], [64, 1, 30], 3, 1, 128, 64, 16, "hnd"),
    ([9001, 30], [8, 8], 12, 2, 128, 128, 64, "nhd"),
    ([5000] * 3, [2] * 3, 48, 1, 64, 16, 16, "nhd"),
]


@pytest.mark.parametrize("case", DECODES)
def test_decode(pm, case):
    c = Decode(*case)
    o, lse, ws = c.run(pm)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse, str(case[2:]))
    # again on the same workspace (its counters are as they were): the same bits
    o2, lse2, _ = c.run(pm, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("held,new,Hq,Hk,ps,bs,layout", [
    ([1], [1], 2, 2, 1, 1, "nhd"),
    ([0, 5, 0, 0, 130, 0], [1, 1, 0, 1, 1, 1], 6, 2, 4, 2, "hnd"),
    ([257, 700, 33], [1] * 3, 80, 2, 64, 64, "nhd"),
    ([9001, 1, 4000], [1] * 3, 5, 5, 1, 1, "shared"),
    ([9001, 1, 4000, 64], [3, 1, 4, 2], 9, 3, 128, 32, "nhd"),
    ([130, 200, 65], [64, 1, 30], 4, 4, 32, 32, "hnd"),
    ([33001], [4], 16, 2, 64, 64, "nhd"),
    ([(i * 131) % 1200 for i in range(170)], [2] * 170, 10, 5, 16, 16, "nhd"),
])
def test_decode_of_paired_heads(pm, held, new, Hq, Hk, ps, bs, layout):
    """64-wide heads two at a time, which calls take whose page list has room for more than lies in
    L2; an odd last head has no partner."""
    c = Decode(held, new, Hq, Hk, 64, ps, bs, layout)
    alone = c.run(pm)
    c.pages.indices = torch.cat([c.pages.indices, torch.full((1 << 22,), 1 << 30, dtype=torch.int32, device=DEV)])
    o, lse, ws = c.run(pm)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse)
    c.check(*alone[:2])
    o2, lse2, _ = c.run(pm, ws=ws)
    live = lse.isfinite()
    assert torch.equal(o[live], o2[live]) and torch.equal(lse[live], lse2[live])


@pytest.mark.parametrize("new", [1, 3])
def test_decode_many_requests(pm, new):
    """More requests than a CTA scans at once, empty ones among them; fp32 outputs, padding."""
    held = [(i * 37) % 90 for i in range(700)]
    c = Decode(held, [new if i % 11 else 0 for i in range(700)], 4, 2, 64, 8, 8, pad=7)
    o, lse, ws = c.run(pm, torch.float32)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse, "700 requests")


@pytest.mark.parametrize("n,new,Hq,Hk,D", [
    (33001, 1, 32, 1, 64), (65001, 1, 8, 1, 128), (33001, 4, 8, 1, 64), (33001, 4, 8, 1, 128), (33001, 2, 1, 1, 128),
])
def test_decode_one_request_over_all_spans(pm, n, new, Hq, Hk, D):
    c = Decode([n], [new], Hq, Hk, D, 64, 64)
    o, lse, ws = c.run(pm)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse)
    o2, lse2, _ = c.run(pm, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,Hk,D,new", [(4, 1, 128, 1), (5, 1, 64, 3), (32, 1, 128, 2), (32, 1, 64, 1)])
@pytest.mark.parametrize("held", [[40001] + [i % 5 for i in range(199)], [(i * 131) % 1200 for i in range(170)]])
def test_decode_more_units_than_sms(pm, held, Hq, Hk, D, new):
    c = Decode(held, [new] * len(held), Hq, Hk, D, 16, 16)
    o, lse, ws = c.run(pm)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse)


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 1)])
def test_decode_scales_far_apart(pm, D, bs):
    """Blocks whose scales differ by 2^20 on both sides, zero scales over zero codes, and scales
    that are no powers of two."""
    held = [200, 1, 77]
    c = Decode(held, [1, 1, 2], 4, 1, D, 16, bs)
    g = blk.gen(5, DEV)
    shape = c.vs.shape
    c.vs.copy_(torch.where(c.vs.isnan(), c.vs, torch.exp2(torch.rand(shape, generator=g, device=DEV) * 20 - 10)))
    c.ks.copy_(torch.where(c.ks.isnan(), c.ks, c.ks * (1 + torch.rand(shape, generator=g, device=DEV))))
    zero = c.pages.where(0, 32, 48)
    for cache, scale in ((c.kc, c.ks), (c.vc, c.vs)):
        cache.view(torch.uint8)[zero] = 0
        scale[zero[0], zero[1] // bs] = 0
    o, lse, ws = c.run(pm)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse)


def test_decode_does_not_depend_on_the_slots_behind(pm):
    """Poison in the last page's tail, in other pages and in their scales is never read (the
    caches hold NaN there); infinite scales there change nothing either."""
    c = Decode([37, 130], [1, 4], 8, 2, 128, 128, 32)
    o, lse, ws = c.run(pm)
    c.ks.copy_(torch.where(c.ks.isnan(), math.inf, c.ks))
    c.vs.copy_(torch.where(c.vs.isnan(), -math.inf, c.vs))
    o2, lse2, _ = c.run(pm, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_device_errors(pm):
    c = Decode([40, 33, 20], [1, 2, 1], 4, 2, 64, 16, 16, pad=3)
    good, lse_good, ws = c.run(pm)
    rows = slice(1, 3)                         # request 1
    others = [0, 3]
    for what in ("tokens", "long", "list"):
        keep = c.qo.clone(), c.pages.indptr.clone()
        if what == "tokens":
            c.qo[2] = 900
        elif what == "long":
            c.new = [1, 1, 1]                  # max_seqlen_q 1 with two tokens in request 1
        else:
            c.pages.indptr[2] = 1 << 20        # requests 1 and 2 make no sense: empty
        o, lse, _ = c.run(pm, ws=ws)
        assert pm.mla_check_error(ws) == 5
        assert torch.equal(o[0], good[0])
        if what == "list":
            assert (o[rows] == 0).all() and torch.isneginf(lse[rows]).all() and (o[3] == 0).all()
        else:
            assert o[rows].isnan().all() and lse[rows].isnan().all()
        c.qo, c.pages.indptr = keep
        c.new = [1, 2, 1]
    bad = c.pages.indices.clone()
    bad[0] = c.pages.pool                      # request 0's first page: reads as zeros
    c.pages.indices, keep = bad, c.pages.indices
    o, lse, _ = c.run(pm, ws=ws)
    assert pm.mla_check_error(ws) == 5
    assert not o[:4].isnan().any() and torch.equal(o[1:4], good[1:4])
    c.pages.indices = keep
    o, lse, _ = c.run(pm, ws=ws)
    assert pm.mla_check_error(ws) == 0 and torch.equal(o[:4], good[:4])
    assert o[others].isfinite().all()


def test_decode_shares_a_workspace_with_the_plain_decode(pm):
    c = Decode([30001], [1], 8, 1, 128, 64, 64)
    ws = pm.make_gqa_block_decode_workspace(8, 1, 128, 1, DEV)
    o, lse, _ = c.run(pm, ws=ws)
    one = torch.tensor(0.02, device=DEV)
    args = (c.q, c.kc, c.vc, torch.empty_like(o), c.pages.indptr, c.pages.indices, c.pages.last, c.sm, one, one)
    pm.mla_gqa_decode(*args, workspace=ws)
    first = args[3].clone()
    o2, lse2, _ = c.run(pm, ws=ws)
    pm.mla_gqa_decode(*args, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(first, args[3])
    assert pm.mla_check_error(ws) == 0


# More than 16 query rows a KV head (its own kernel where the cache's layout allows it).
@pytest.mark.parametrize("held,new,Hq,Hk,D,ps,bs,layout", [
    ([1, 0, 127, 128, 129, 255, 300], [1] * 7, 20, 1, 128, 8, 8, "nhd"),
    ([700, 3, 64, 0], [3] * 4, 18, 3, 64, 8, 4, "nhd"),                # the last head has no partner
    ([700, 3, 64], [3] * 3, 18, 3, 64, 16, 16, "hnd"),
    ([700, 3], [2] * 2, 24, 2, 64, 16, 16, "shared"),
    ([700, 3], [2] * 2, 24, 2, 128, 16, 16, "shared"),
    ([4100, 17], [5, 2], 48, 4, 128, 1024, 128, "hnd"),
    ([300], [64], 8, 1, 128, 256, 64, "nhd"),
    ([300, 70], [64, 33], 4, 2, 64, 128, 128, "nhd"),
    ([5, 300, 40], [64, 64, 50], 2, 1, 128, 16, 16, "nhd"),            # queries that see nothing
    ([5, 300, 40], [64, 64, 50], 4, 4, 64, 8, 8, "nhd"),
    ([2001] * 5, [2] * 5, 40, 2, 128, 4, 4, "nhd"),
    ([65001], [4], 16, 2, 128, 64, 64, "nhd"),
    ([33001], [4], 16, 2, 64, 64, 64, "nhd"),
    ([(i * 131) % 1200 for i in range(170)], [2] * 170, 40, 2, 128, 16, 16, "nhd"),
    ([40001] + [i % 7 for i in range(199)], [1] * 200, 34, 2, 64, 32, 32, "nhd"),
])
def test_decode_of_many_rows(pm, held, new, Hq, Hk, D, ps, bs, layout):
    c = Decode(held, new, Hq, Hk, D, ps, bs, layout, pad=2)
    o, lse, ws = c.run(pm, torch.float32)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse, "", blk.LOST_MANY)
    o2, lse2, _ = c.run(pm, torch.float32, ws=ws)
    n = sum(new)
    assert torch.equal(o[:n], o2[:n]) and torch.equal(lse[:n], lse2[:n])


@pytest.mark.parametrize("rows", [4, 32])
def test_decode_of_one_large_score_among_many_small(pm, rows):
    """The first position has e^14 times the weight of each of 60,000 others, whose 4 % of the mass
    (weights of 2^-20 of the largest) are all of the output that is not zero."""
    c = Decode([60001], [1], rows, 1, 128, 64, 64)
    page, slot = c.pages.where(0, 0, 60001)
    for cache, code in ((c.kc, 0.0), (c.vc, 1.0)):
        cache.view(torch.uint8)[page, slot] = torch.tensor(code, device=DEV).to(blk.F8).view(torch.uint8)
    c.kc.view(torch.uint8)[page[0], slot[0]] = torch.tensor(20.0, device=DEV).to(blk.F8).view(torch.uint8)
    c.vc.view(torch.uint8)[page[0], slot[0]] = 0
    c.ks[page, slot // 64] = 2.0 ** -4
    c.vs[page, slot // 64] = 1.0
    c.q.fill_(1.0)
    o, lse, ws = c.run(pm, torch.float32)
    assert pm.mla_check_error(ws) == 0
    want = 60000 / (60000 + math.exp(128 ** 0.5 * 20 / 16))
    # each weight, 2^-20.4 of the largest: rounded to a multiple of 2^-24 (by 2^-25 at most)
    assert 0.04 < want < 0.05 and ((o.double() - want).abs() / want).max().item() < 2.0 ** -25 * 2.0 ** 20.5 + 2.0 ** -10
    c.check(o, lse, "", blk.LOST_MANY)


@pytest.mark.parametrize("Hq,Hk,D", [(40, 2, 128), (36, 2, 64)])
def test_decode_of_many_rows_reads_only_its_lists(pm, Hq, Hk, D):
    """Poison behind the lists, infinite scales there, a page that is not in the cache, a list that
    makes no sense: as with few rows."""
    c = Decode([37, 300, 130], [1, 3, 2], Hq, Hk, D, 16, 16)
    good, lse_good, ws = c.run(pm)
    c.check(good, lse_good, "", blk.LOST_MANY)
    c.ks.copy_(torch.where(c.ks.isnan(), math.inf, c.ks))
    c.vs.copy_(torch.where(c.vs.isnan(), -math.inf, c.vs))
    o, lse, _ = c.run(pm, ws=ws)
    assert pm.mla_check_error(ws) == 0 and torch.equal(o, good) and torch.equal(lse, lse_good)
    for wrong in (c.pages.pool, -1, 1 << 30):
        keep = c.pages.indices
        c.pages.indices = keep.clone()
        c.pages.indices[1] = wrong             # request 0's second page: zeros
        o, lse, _ = c.run(pm, ws=ws)
        c.pages.indices = keep
        assert pm.mla_check_error(ws) == 5
        assert torch.equal(o[1:], good[1:]) and o.isfinite().all()
        k, v = (blk.values(c.pages, 0, x, s).double() for x, s in ((c.kc, c.ks), (c.vc, c.vs)))
        k[16:32] = 0
        v[16:32] = 0
        q = c.q[0].double().view(Hk, Hq // Hk, D)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * c.sm, -1)
        want = torch.einsum("hgn,nhd->hgd", p, v).reshape(Hq, D)
        most = torch.einsum("hgn,nhd->hgd", p, v.abs()).reshape(Hq, D)
        assert ((o[0].double() - want).abs() <= most * 2.0 ** -7 + 1e-6).all()
    keep = c.pages.indptr.clone()
    c.pages.indptr[2] = 1 << 20
    o, lse, _ = c.run(pm, ws=ws)
    assert pm.mla_check_error(ws) == 5
    assert torch.equal(o[0], good[0]) and (o[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    c.pages.indptr = keep
    o, lse, _ = c.run(pm, ws=ws)
    assert pm.mla_check_error(ws) == 0 and torch.equal(o, good)


def test_decode_of_many_rows_in_a_graph(pm):
    """Captured once, replayed after lengths, pages and rows have changed in place."""
    a, b = (Decode(held, [2, 2, 2], 40, 2, 128, 16, 16, seed=3) for held in ([500, 40, 3000], [2, 3000, 530]))
    ws = pm.make_gqa_block_decode_workspace(40, 2, 128, 2, DEV)
    want = [x.run(pm, ws=ws)[:2] for x in (a, b)]
    assert a.pages.indices.shape == b.pages.indices.shape and a.kc.shape == b.kc.shape
    o, lse = (torch.empty_like(x) for x in want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pm.mla_gqa_block_decode(a.q, a.kc, a.vc, a.ks, a.vs, o, a.qo, a.pages.indptr, a.pages.indices,
                                a.pages.last, 2, a.sm, lse, ws)
    g.replay()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    for x, y in ((a.q, b.q), (a.kc.view(torch.uint8), b.kc.view(torch.uint8)),
                 (a.vc.view(torch.uint8), b.vc.view(torch.uint8)), (a.ks, b.ks), (a.vs, b.vs),
                 (a.pages.indptr, b.pages.indptr), (a.pages.indices, b.pages.indices), (a.pages.last, b.pages.last)):
        x.copy_(y)
    g.replay()
    assert torch.equal(o, want[1][0]) and torch.equal(lse, want[1][1])
    assert pm.mla_check_error(ws) == 0


@pytest.mark.parametrize("new", [1, 3])       # 8 rows a KV head, and 24
@pytest.mark.parametrize("D", [64, 128])
def test_decode_keeps_heads_apart(pm, D, new):
    """NaN codes, NaN scales and infinite queries of one head leave the others' bits as they were."""
    c = Decode([300, 2000], [new, new], 24, 3, D, 16, 16)
    c.pages.indices = torch.cat([c.pages.indices, torch.full((1 << 22,), 1 << 30, dtype=torch.int32, device=DEV)])
    good, lse_good, ws = c.run(pm)
    page, slot = c.pages.where(1, 70, 90)
    group = lambda x, h: x.view(2 * new, 3, 8, -1)[:, h]
    for h in range(3):
        others = [x for x in range(3) if x != h]
        for what in ("k code", "v code", "k scale", "v scale", "q"):
            if what == "q":
                x, at, bad = c.q, (slice(None), slice(8 * h, 8 * h + 8)), math.inf
            else:
                x = {"k code": c.kc, "v code": c.vc, "k scale": c.ks, "v scale": c.vs}[what]
                at, bad = ((page, slot, h), 0x7F) if "code" in what else ((page, 0, h), math.nan)
                x = x.view(torch.uint8) if "code" in what else x
            keep = x[at].clone()
            x[at] = bad
            o, lse, _ = c.run(pm, ws=ws)
            x[at] = keep
            for g in others:
                assert torch.equal(group(o, g), group(good, g)) and torch.equal(group(lse, g), group(lse_good, g)), (what, h, g)
    o, lse, _ = c.run(pm, ws=ws)
    assert torch.equal(o, good) and torch.equal(lse, lse_good) and pm.mla_check_error(ws) == 0


def test_decode_of_many_rows_and_requests(pm):
    """More requests than a CTA scans at once, empty ones among them."""
    held = [(i * 37) % 290 for i in range(900)]
    c = Decode(held, [2 if i % 11 else 0 for i in range(900)], 20, 2, 64, 8, 8, pad=7)
    o, lse, ws = c.run(pm, torch.float32)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse, "900 requests", blk.LOST_MANY)

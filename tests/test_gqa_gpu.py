"""The per-head cache's append and the attention of one new token over it, against fp64."""
import math

import pytest
import torch

from tests import gqa_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).bfloat16()


def _cache(pages, ps, hk, d, fp8, layout, poison=True):
    """A pair of empty caches: slots outside heads ("nhd"), heads outside slots ("hnd"), or
    keys and values interleaved in one tensor of wider rows ("shared")."""
    kind = torch.uint8 if fp8 else torch.bfloat16
    if layout == "shared":
        both = torch.zeros(pages, 2, ps, hk, d + 16, dtype=kind, device=DEV)
        k, v = both[:, 0, :, :, :d], both[:, 1, :, :, :d]
    elif layout == "hnd":
        k, v = (torch.zeros(pages, hk, ps, d, dtype=kind, device=DEV).transpose(1, 2) for _ in range(2))
    else:
        k, v = (torch.zeros(pages, ps, hk, d, dtype=kind, device=DEV) for _ in range(2))
    for t in (k, v):
        t.fill_(0x7F if fp8 else math.nan)
    if fp8:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return k, v


def _table(max_pos, r):
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / r)
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _rows(cache, slots, ps):
    """The entries at some slots, fp64 (T, Hk, D)."""
    bits = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    got = bits[slots.long() // ps, slots.long() % ps]
    return (got.view(torch.float8_e4m3fn).float() if cache.dtype == torch.float8_e4m3fn else got).double()


@pytest.mark.parametrize("T,Hq,Hk,D,R,neox,ps,fp8,layout", [
    (1, 1, 1, 64, 16, 0, 1, False, "nhd"),
    (5, 8, 2, 128, 128, 1, 16, False, "nhd"),
    (5, 8, 2, 128, 128, 0, 16, True, "nhd"),
    (77, 14, 2, 64, 32, 1, 32, True, "hnd"),
    (77, 25, 5, 64, 64, 0, 4, False, "shared"),
    (130, 12, 12, 128, 96, 1, 128, True, "shared"),
    (1031, 16, 1, 128, 64, 1, 1024, False, "hnd"),
])
def test_append(pm, T, Hq, Hk, D, R, neox, ps, fp8, layout):
    g = _gen(T + D)
    # q, k and v as views of one projection, the outputs of wider rows
    qkv = _randn(g, T, (Hq + 2 * Hk) * D + 8)
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    v = qkv[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(T, Hk, D)
    pages = -(-2 * T // ps) + 1
    kc, vc = _cache(pages, ps, Hk, D, fp8, layout)
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T].to(torch.int32)
    if T > 3:
        slots[3] = -1
    pos = torch.randint(0, 500, (T,), generator=g, device=DEV, dtype=torch.int32)
    cs = _table(500, R)
    ks, vs = (torch.tensor(0.02, device=DEV), torch.tensor([0.015], device=DEV)) if fp8 else (None, None)
    q_out = torch.full((T, Hq, D + 8), math.nan, dtype=torch.bfloat16, device=DEV)[:, :, :D]
    k_out = torch.full((T, Hk, D), math.nan, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pm.mla_gqa_rope_and_cache(q, k, v, pos, cs, neox, slots, q_out, kc, vc, err, ks, vs, k_out)
    assert err.item() == 0
    live = slots >= 0
    for got, x in ((q_out, q), (k_out, k)):
        want, mag = ref.rotate(x, cs, pos, neox)
        off = (got.double() - want).abs()
        # two products and their sum in fp32, then one rounding to bf16
        assert (off <= ref.BF16 * want.abs() + 3 * ref.F32 * mag).all()
        assert torch.equal(got[..., R:], x[..., R:])
    for cache, x, s, turned in ((kc, k, ks, True), (vc, v, vs, False)):
        want, mag = ref.rotate(x, cs, pos, neox) if turned else (x.double(), x.double().abs())
        want, mag = want[live], mag[live]
        got = _rows(cache, slots[live], ps)
        if fp8:
            want, mag = (want / s.double()).clamp(-448, 448), mag / s.double()
            # half a step of e4m3 (2^-10 among its subnormals); the fp32 quotient's own error
            # can move a value across a border between two codes
            bound = ref.E4M3 * want.abs() + 2.0 ** -10 + 5 * ref.F32 * mag
        else:
            bound = ref.BF16 * want.abs() + 3 * ref.F32 * mag
        assert ((got - want).abs() <= bound).all()
    # nothing but the mapped slots was written
    for cache in (kc, vc):
        bits = cache.view(torch.uint8) if fp8 else cache
        untouched = torch.ones(pages * ps, dtype=torch.bool, device=DEV)
        untouched[slots[live].long()] = False
        rest = bits.reshape(pages * ps, Hk, D)[untouched]
        assert ((rest == 0x7F) if fp8 else rest.isnan()).all()


@pytest.mark.parametrize("scale", [None, 1.0, 0.0237, 3e-13, 2.0 ** 41, 1e-20])
@pytest.mark.parametrize("neox", [0, 1])
def test_append_is_exact(pm, neox, scale):
    """The definition's fp32 arithmetic, every operation rounded on its own, bit for bit (torch's
    elementwise operations round so), for scales on both sides of the quotients' two ways."""
    T, H, D, R = 5000, 2, 128, 96
    g = _gen(11 + neox)
    q, k, v = _randn(g, T, H, D), _randn(g, T, H, D), _randn(g, T, H, D, std=3.0)
    if scale:
        k, v = (x.float().mul(min(scale, 1e36) * 40).bfloat16() for x in (k, v))
        v[0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 3e38, -3e38, 1e-38], device=DEV).bfloat16()
    pos = torch.randint(0, 70000, (T,), generator=g, device=DEV, dtype=torch.int32)
    cs = _table(70000, R)
    kc, vc = _cache(T, 1, H, D, scale is not None, "nhd")
    s = None if scale is None else torch.tensor(scale, device=DEV)
    slots, err = torch.arange(T, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.empty_like(q)
    pm.mla_gqa_rope_and_cache(q, k, v, pos, cs, neox, slots, q_out, kc, vc, err, s, s)
    row = cs[pos.long()][:, None]
    c, sn = row[..., :R // 2], row[..., R // 2:]

    def turned(x):
        x = x.float()
        a, b = (x[..., :R // 2], x[..., R // 2:R]) if neox else (x[..., 0:R:2], x[..., 1:R:2])
        u, w = a * c - b * sn, b * c + a * sn
        front = torch.cat([u, w], -1) if neox else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([front, x[..., R:]], -1)

    def bits(x):
        return x.view(torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16)

    assert torch.equal(bits(q_out), bits(turned(q).bfloat16()))
    for cache, x in ((kc, turned(k)), (vc, v.float())):
        want = x.bfloat16() if scale is None else (x / s).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = cache[:, 0]
        nan = want.float().isnan()
        assert torch.equal(got.float().isnan(), nan)
        assert torch.equal(bits(got)[~nan], bits(want)[~nan])


@pytest.mark.parametrize("neox", [0, 1])
def test_append_in_place(pm, neox):
    g = _gen(3)
    q, k, v = _randn(g, 9, 6, 64), _randn(g, 9, 2, 64), _randn(g, 9, 2, 64)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    slots = torch.arange(9, dtype=torch.int32, device=DEV)
    cs, err = _table(16, 64), torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for in_place in (False, True):
        q1, k1 = q.clone(), k.clone()
        kc, vc = _cache(2, 16, 2, 64, False, "nhd")
        qo, ko = (q1, k1) if in_place else (torch.empty_like(q), torch.empty_like(k))
        pm.mla_gqa_rope_and_cache(q1, k1, v, pos, cs, neox, slots, qo, kc, vc, err, k_out=ko)
        outs.append((qo, ko, kc.view(torch.int16), vc.view(torch.int16)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_append_saturates_and_keeps_nan(pm):
    T, D = 2, 64
    q = torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV)
    v[0, 0, :4] = torch.tensor([1e9, -1e9, math.nan, 3.0], device=DEV).bfloat16()
    k[1, 0, 60] = 5e4
    kc, vc = _cache(1, 2, 1, D, True, "nhd")
    one = torch.ones((), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    i = torch.arange(T, dtype=torch.int32, device=DEV)
    pm.mla_gqa_rope_and_cache(q, k, v, i, _table(4, 16), 1, i, torch.empty_like(q), kc, vc, err, one, one)
    got = vc.float()[0, 0, 0]
    assert got[0] == 448 and got[1] == -448 and got[2].isnan() and got[3] == 3
    assert kc.float()[0, 1, 0, 60] == 448


def test_append_flags_bad_slots_and_positions(pm):
    T, D = 4, 64
    g = _gen(8)
    q, k, v = _randn(g, T, 2, D), _randn(g, T, 2, D), _randn(g, T, 2, D)
    kc, vc = _cache(2, 4, 2, D, False, "nhd")
    slots = torch.tensor([0, 8, 2, 3], dtype=torch.int32, device=DEV)      # 8: past the cache
    pos = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full_like(q, math.nan)
    pm.mla_gqa_rope_and_cache(q, k, v, pos, _table(4, 32), 1, slots, q_out, kc, vc, err)
    assert err.item() == 64
    assert not q_out.isnan().any()
    for bad in (-1, 4):
        err.zero_()
        q_out.fill_(math.nan)
        kc, vc = _cache(2, 4, 2, D, False, "nhd")
        pos[2] = bad
        slots[1] = 1
        pm.mla_gqa_rope_and_cache(q, k, v, pos, _table(4, 32), 1, slots, q_out, kc, vc, err)
        assert err.item() == 1
        assert q_out[2, :, :32].isnan().all() and not q_out[2, :, 32:].isnan().any()
        assert not q_out[[0, 1, 3]].isnan().any()
        assert kc[0, 2, :, :32].isnan().all() and torch.equal(vc[0, 2], v[2])


def _decode_case(lens, Hq, Hk, D, ps, fp8, layout="nhd", seed=0, std=1.5):
    g = _gen(seed + sum(lens) + 17 * D + ps)
    n_pages = [-(-n // ps) for n in lens]
    total = sum(n_pages)
    pool = total + 3
    kc, vc = _cache(pool, ps, Hk, D, fp8, layout)
    ids = torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32)
    at, keys = 0, []
    for n, p in zip(lens, n_pages):
        x = [torch.randn(p * ps, Hk, D, generator=g, device=DEV) * (50 if fp8 else 1) for _ in range(2)]
        x = [y.clamp(-448, 448).to(kc.dtype) for y in x]
        mine = ids[at:at + p].long()
        for cache, y in zip((kc, vc), x):
            if fp8:
                cache, y = cache.view(torch.uint8), y.view(torch.uint8)
            y[n:] = 0x7F if fp8 else math.nan              # the last page's tail stays poison
            cache[mine] = y.view(p, ps, Hk, D)
        keys.append([y[:n] for y in x])
        at += p
    indptr = torch.tensor([0] + list(torch.tensor(n_pages).cumsum(0)), dtype=torch.int32, device=DEV)
    last = torch.tensor([n - (p - 1) * ps if n else 1 for n, p in zip(lens, n_pages)], dtype=torch.int32,
                        device=DEV)
    q = _randn(g, len(lens), Hq, D, std=std)
    tail = torch.full((5,), 1 << 30, dtype=torch.int32, device=DEV)        # never read
    return dict(q=q, kc=kc, vc=vc, indptr=indptr, idx=torch.cat([ids, tail]), last=last, keys=keys,
                ks=torch.tensor(0.02, device=DEV) if fp8 else None,
                vs=torch.tensor(0.015, device=DEV) if fp8 else None, sm=D ** -0.5)


def _decode_ref(c, b):
    q = c["q"][b].double()
    k, v = (x.float().double() for x in c["keys"][b])
    Hk = c["kc"].shape[2]
    G = q.shape[0] // Hk
    if c["ks"] is not None:
        k, v = k * c["ks"].double(), v * c["vs"].double()
    n = k.shape[0]
    out = [ref.attend(q[h * G:(h + 1) * G], k[:, h], v[:, h], c["sm"],
                      torch.full((G,), n, device=DEV)) for h in range(Hk)]
    return [torch.cat(x) for x in zip(*out)]


def _run_decode(pm, c, o_dtype=torch.bfloat16, ws=None, **kw):
    B, Hq, D = c["q"].shape
    o = torch.full((B, Hq, D), math.nan, dtype=o_dtype, device=DEV)
    lse = torch.full((B, Hq), math.nan, device=DEV)
    ws = pm.mla_gqa_decode(c["q"], c["kc"], c["vc"], o, c["indptr"], c["idx"], c["last"], c["sm"],
                           c["ks"], c["vs"], lse, ws, **kw)
    return o, lse, ws


def _check_decode(c, o, lse, what):
    fp8 = c["ks"] is not None
    for b in range(o.shape[0]):
        n = c["keys"][b][0].shape[0]
        ref.check(o[b], lse[b], _decode_ref(c, b), n, c["q"].shape[2], ref.F16 if fp8 else ref.BF16,
                  ref.F32 if o.dtype == torch.float32 else ref.BF16, f"{what}, request {b} of {n}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hk,D,ps,layout", [
    ([1], 1, 1, 64, 1, "nhd"),
    ([1, 2, 15, 16, 17, 31, 33, 63, 64, 65], 8, 2, 128, 16, "nhd"),
    ([0, 5, 0, 0, 130, 0], 6, 2, 64, 4, "hnd"),
    ([0, 0], 4, 2, 128, 16, "nhd"),
    ([300, 7, 129], 9, 1, 128, 2, "shared"),
    ([2049, 1023], 16, 1, 64, 1024, "nhd"),
    ([511, 40, 1], 33, 1, 128, 32, "hnd"),
    ([257, 700], 80, 2, 64, 64, "nhd"),
    ([777], 32, 2, 128, 128, "shared"),
    ([9001, 1, 4000], 5, 5, 128, 1, "nhd"),
    ([20011], 64, 8, 128, 128, "nhd"),
])
def test_decode(pm, lens, Hq, Hk, D, ps, fp8, layout):
    c = _decode_case(lens, Hq, Hk, D, ps, fp8, layout)
    o, lse, ws = _run_decode(pm, c)
    assert pm.mla_check_error(ws) == 0
    _check_decode(c, o, lse, f"{Hq}/{Hk} heads")
    # again on the same workspace (its counters are as they were): the same bits
    o2, lse2, _ = _run_decode(pm, c, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_requests(pm, fp8):
    """More requests than a CTA scans at once, empty ones among them; fp32 outputs."""
    lens = [(i * 37) % 90 for i in range(700)]
    c = _decode_case(lens, 4, 2, 64, 8, fp8)
    o, lse, ws = _run_decode(pm, c, torch.float32)
    assert pm.mla_check_error(ws) == 0
    _check_decode(c, o, lse, "700 requests")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hq,Hk,D", [
    (33001, 32, 1, 64),        # one unit over every span: as many pieces as there are CTAs
    (65001, 32, 1, 64),
    (33001, 8, 1, 64),
    (33001, 32, 1, 128),
])
def test_decode_one_unit_over_all_spans(pm, n, Hq, Hk, D, fp8):
    c = _decode_case([n], Hq, Hk, D, 64, fp8)
    o, lse, ws = _run_decode(pm, c)
    assert pm.mla_check_error(ws) == 0
    _check_decode(c, o, lse, f"{Hq}/{Hk} heads of {D}")
    o2, lse2, _ = _run_decode(pm, c, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (5, 1, 64), (16, 1, 128), (12, 1, 64), (32, 1, 128), (32, 1, 64)])
@pytest.mark.parametrize("lens", [
    [40001] + [i % 5 for i in range(199)],         # one unit over nearly all spans
    [(i * 131) % 1200 for i in range(170)],
])
def test_decode_more_units_than_sms(pm, lens, Hq, Hk, D, fp8):
    c = _decode_case(lens, Hq, Hk, D, 32, fp8)
    o, lse, ws = _run_decode(pm, c)
    assert pm.mla_check_error(ws) == 0
    _check_decode(c, o, lse, f"{Hq}/{Hk} heads of {D}")
    o2, lse2, _ = _run_decode(pm, c, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_one_strong_key(pm, fp8):
    """One key takes nearly all of the weight, first, last or amid many; the rest is what
    the running maximum has to drop."""
    n, D = 4099, 128
    for at in (0, 1, 2000, n - 1):
        c = _decode_case([n], 8, 1, D, 16, fp8, seed=at)
        k = c["keys"][0][0]
        q0 = c["q"][0, 0].float()
        strong = (q0 * (100.0 if fp8 else 4.0)).clamp(-448, 448)
        page, slot = int(c["idx"][at // 16]), at % 16
        if fp8:
            c["kc"].view(torch.uint8)[page, slot, 0] = strong.to(torch.float8_e4m3fn).view(torch.uint8)
            k.view(torch.uint8)[at, 0] = strong.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            c["kc"][page, slot, 0] = strong.bfloat16()
            k[at, 0] = strong.bfloat16()
        o, lse, _ = _run_decode(pm, c)
        _check_decode(c, o, lse, f"strong key at {at}")


def test_decode_extreme_queries(pm):
    """e4m3 caches multiply in f16: queries far outside f16's range still come out."""
    for std in (1e-30, 1e-6, 1e8):
        c = _decode_case([100, 333], 8, 2, 64, 16, True, std=std)
        if std > 1:
            c["sm"] = 1e-8
        o, lse, _ = _run_decode(pm, c)
        _check_decode(c, o, lse, f"queries of size {std}")


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_scales(pm, fp8):
    """Softmax scales of zero (a plain mean), below zero and large."""
    for sm in (0.0, -0.2, 2.0):
        c = _decode_case([1, 400, 3000], 8, 2, 64, 16, fp8)
        c["sm"] = sm
        o, lse, _ = _run_decode(pm, c)
        _check_decode(c, o, lse, f"sm_scale {sm}")


def test_decode_shapes_share_a_workspace(pm):
    shapes = [([5000, 17], 8, 1, 128, 16, False), ([3000] * 3, 40, 1, 128, 64, True),
              ([7000], 16, 2, 64, 128, False), ([5000, 17], 8, 1, 128, 16, True)]
    n = max(pm.mla_get_gqa_decode_workspace_size(len(s[0]), s[1], s[2], s[3]) for s in shapes)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for lens, Hq, Hk, D, ps, fp8 in shapes:
            c = _decode_case(lens, Hq, Hk, D, ps, fp8)
            o, lse, _ = _run_decode(pm, c, ws=ws)
            _check_decode(c, o, lse, f"{Hq}/{Hk} of {D}")
    assert pm.mla_check_error(ws) == 0


def test_decode_infinite_scores(pm):
    """A key of -inf scores drops out; NaN in an attended key or value reaches the row."""
    c = _decode_case([40], 4, 1, 64, 8, False)
    c["q"].abs_()
    page = int(c["idx"][0])
    c["kc"][page, 3, 0] = -math.inf
    k, v = c["keys"][0]
    o, lse, _ = _run_decode(pm, c)
    keep = torch.arange(40, device=DEV) != 3
    c["keys"][0] = [k[keep], v[keep]]
    _check_decode(c, o, lse, "a key at -inf")
    c["vc"][page, 5, 0, 7] = math.nan
    o, _, _ = _run_decode(pm, c)
    assert o[0, :, 7].isnan().all() and not o[0, :, :7].isnan().any()
    c["kc"][:, :, 0] = -math.inf              # nothing has weight
    o, lse, _ = _run_decode(pm, c)
    assert lse.isneginf().all()


def test_decode_bad_tables(pm):
    c = _decode_case([40, 50, 60], 4, 2, 64, 16, False)
    good_o, good_lse, ws = _run_decode(pm, c)
    idx, indptr = c["idx"].clone(), c["indptr"].clone()
    c["idx"] = idx.clone()
    c["idx"][4] = 10 ** 6                     # request 1's second page
    o, lse, ws = _run_decode(pm, c, ws=ws)
    assert pm.mla_check_error(ws) == 5
    assert torch.equal(o[[0, 2]], good_o[[0, 2]]) and torch.isfinite(o).all()
    c["idx"] = idx
    c["indptr"] = indptr.clone()
    c["indptr"][3] = 10 ** 6                  # leaves kv_indices: request 2 counts as empty
    o, lse, ws = _run_decode(pm, c, ws=ws)
    assert pm.mla_check_error(ws) == 5
    assert torch.equal(o[:2], good_o[:2]) and (o[2] == 0).all() and lse[2].isneginf().all()
    c["indptr"] = indptr
    o, lse, ws = _run_decode(pm, c, ws=ws)
    assert pm.mla_check_error(ws) == 0
    assert torch.equal(o, good_o) and torch.equal(lse, good_lse)


def test_decode_far_pages(pm):
    """Entries past 2^32 bytes into a cache."""
    D, Hk, ps, pages = 128, 8, 128, 40000            # 10.5 GB of keys
    kc = torch.empty(pages, ps, Hk, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty(pages, ps, Hk, D, dtype=torch.bfloat16, device=DEV)
    g = _gen(1)
    ids = torch.tensor([39999, 3, 20480], dtype=torch.int32, device=DEV)
    n = 2 * ps + 77
    k, v = _randn(g, 3 * ps, Hk, D), _randn(g, 3 * ps, Hk, D)
    for i, page in enumerate(ids.tolist()):
        kc[page], vc[page] = k[i * ps:(i + 1) * ps], v[i * ps:(i + 1) * ps]
    c = dict(q=_randn(g, 1, 16, D), kc=kc, vc=vc, indptr=torch.tensor([0, 3], dtype=torch.int32, device=DEV),
             idx=ids, last=torch.tensor([77], dtype=torch.int32, device=DEV), keys=[[k[:n], v[:n]]],
             ks=None, vs=None, sm=D ** -0.5)
    o, lse, ws = _run_decode(pm, c)
    assert pm.mla_check_error(ws) == 0
    _check_decode(c, o, lse, "far pages")


def test_decode_on_another_stream_and_in_a_graph(pm):
    c = _decode_case([900, 33], 8, 2, 128, 16, False)
    want_o, want_lse, _ = _run_decode(pm, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse, ws = _run_decode(pm, c)
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse)
    o.fill_(math.nan)
    torch.cuda.synchronize()                  # the call below makes its workspace on s, too
    pm.mla_gqa_decode(c["q"], c["kc"], c["vc"], o, c["indptr"], c["idx"], c["last"], c["sm"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, want_o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pm.mla_gqa_decode(c["q"], c["kc"], c["vc"], o, c["indptr"], c["idx"], c["last"], c["sm"],
                          lse_out=lse, workspace=ws)
    for _ in range(3):
        o.fill_(math.nan)
        graph.replay()
        assert torch.equal(o, want_o)
    c["last"][0] = 1                          # 897 positions: the same graph, new lengths
    c["keys"][0] = [x[:897] for x in c["keys"][0]]
    graph.replay()
    _check_decode(c, o, lse, "replayed with another length")

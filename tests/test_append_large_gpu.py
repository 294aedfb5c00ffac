"""The append on both sides of the size from which a thread takes two heads at a time: the same
bytes as the definition's fp32 arithmetic, every operation rounded on its own."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _tokens(Hq, Hk, D, more):
    """The fewest tokens whose items (8-column pairs of words) are four waves of 2,048 threads a
    SM, and `more`."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-sms * 2048 * 4 // ((Hq + 2 * Hk) * (D // 16))) + more


def _bits(x):
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)


def _turned(x, row, R, neox):
    x = x.float()
    c, s = row[..., :R // 2], row[..., R // 2:]
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if neox else (x[..., 0:R:2], x[..., 1:R:2])
    u, w = a * c - b * s, b * c + a * s
    front = torch.cat([u, w], -1) if neox else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([front, x[..., R:]], -1)


def _table(n, R):
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R)
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("neox", [0, 1])
@pytest.mark.parametrize("Hq,Hk,D,R,more", [
    (25, 5, 64, 32, 700),            # odd heads: the last strip of q, k and v holds one
    (25, 5, 64, 64, 0),              # the first size of two heads a thread
    (25, 5, 64, 64, -1),             # the last of one
    (9, 3, 128, 96, 700),
    (8, 1, 128, 128, 300),           # one key head
    (33, 11, 128, 16, 700),          # more items than a block has threads
    (1, 1, 64, 16, 300),
])
def test_append_bytes(pm, Hq, Hk, D, R, more, neox, fp8):
    T = _tokens(Hq, Hk, D, more)
    g = torch.Generator(device=DEV).manual_seed(T)
    ps, max_pos = 16, 5000
    pages = -(-T // ps) + 3
    # views of one projection
    qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=g, device=DEV).bfloat16()
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    v = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
    v[7, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3e38], device=DEV)
    pos = torch.randint(0, max_pos, (T,), generator=g, device=DEV, dtype=torch.int32)
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T].to(torch.int32)
    slots[::5] = -1                            # padding
    cs = _table(max_pos, R)
    ks, vs = (torch.tensor(0.0237, device=DEV), torch.tensor(0.004, device=DEV)) if fp8 else (None, None)
    kind, blank = (torch.uint8, 0x7F) if fp8 else (torch.bfloat16, math.nan)
    caches = [torch.full((pages, ps, Hk, D), blank, dtype=kind, device=DEV) for _ in range(2)]
    if fp8:
        caches = [c.view(torch.float8_e4m3fn) for c in caches]
    q_out = torch.full((T, Hq, D), math.nan, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((T, Hk, D), math.nan, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def expected(n, x, scale):
        """The cache after x's entries."""
        want = torch.full((pages * ps, Hk, D), blank, dtype=kind, device=DEV)
        live = slots >= 0
        new = x[live].bfloat16() if scale is None else \
            (x[live] / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        want[slots[live].long()] = new
        return want.view(pages, ps, Hk, D)

    def same(got, want):
        """Equal bits, NaN anywhere NaN is wanted."""
        got, want = _bits(got), _bits(want)
        nan = (want & 0x7F) == 0x7F if fp8 and want.dtype == torch.uint8 else (want & 0x7FFF) > 0x7F80
        found = (got & 0x7F) == 0x7F if fp8 and want.dtype == torch.uint8 else (got & 0x7FFF) > 0x7F80
        return torch.equal(nan, found) and torch.equal(got[~nan], want[~nan])

    row = cs[pos.long()][:, None]
    tq, tk = _turned(q, row, R, neox), _turned(k, row, R, neox)
    pm.mla_gqa_rope_and_cache(q, k, v, pos, cs, neox, slots, q_out, *caches, err, ks, vs, k_out)
    assert err.item() == 0
    assert same(q_out, tq.bfloat16()) and same(k_out, tk.bfloat16())
    assert same(caches[0], expected("k", tk, ks)) and same(caches[1], expected("v", v.float(), vs))

    # in place over the projection, one token past the cache and one past the table: each is
    # left out and flagged, and nothing else changes
    before = qkv.clone()
    bad_slot, bad_pos = T // 2 + 1, T - 1
    slots[bad_slot], pos[bad_pos] = pages * ps, max_pos
    pos[3] = -1
    for c in caches:
        c.view(kind).fill_(blank)
    pm.mla_gqa_rope_and_cache(q, k, v, pos, cs, neox, slots, q, *caches, err, ks, vs, k)
    assert err.item() == 64 | 1
    known = torch.ones(T, dtype=torch.bool, device=DEV)
    known[bad_pos] = known[3] = False
    q0 = before[:, :Hq * D].view(T, Hq, D)
    k0 = before[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    for got, turned, x in ((q, tq, q0), (k, tk, k0)):
        assert same(got[known], turned[known].bfloat16())
        assert torch.equal(got[~known], x[~known])         # unwritten, and what passes through
    slots[bad_slot] = -1
    want = expected("k", tk, ks)
    for t in (3, bad_pos):                                 # their rotated columns are unwritten
        if slots[t] >= 0:
            want.view(-1, Hk, D)[slots[t].item(), :, :R] = blank
    assert same(caches[0], want) and same(caches[1], expected("v", v.float(), vs))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hk,D,ps", [(3, 64, 16), (2, 128, 1), (1, 128, 4), (2, 64, 128)])
def test_heads_outside_pages(pm, Hk, D, ps, fp8):
    """A cache whose heads are its outermost dim, its pages inside: the append writes and the
    decode reads the same entries as in one of pages outside, and nothing else."""
    T, G, pages, R = 300, 4, -(-300 // ps) + 2, 32
    g = torch.Generator(device=DEV).manual_seed(ps)
    q = torch.randn(T, G * Hk, D, generator=g, device=DEV).bfloat16()
    k, v = (torch.randn(T, Hk, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    ids = torch.randperm(pages, generator=g, device=DEV)[:-(-T // ps)].to(torch.int32)
    slots = (ids.long()[pos.long() // ps] * ps + pos.long() % ps).to(torch.int32)
    cs, err = _table(T, R), torch.zeros(1, dtype=torch.int32, device=DEV)
    scale = torch.tensor(0.02, device=DEV) if fp8 else None
    kind, blank = (torch.uint8, 0x7F) if fp8 else (torch.bfloat16, math.nan)
    got = []
    for shape, order in (((pages, ps, Hk, D), (0, 1, 2, 3)), ((Hk, pages, ps, D), (1, 2, 0, 3))):
        raw = [torch.full(shape, blank, dtype=kind, device=DEV) for _ in range(2)]
        kc, vc = (x.view(torch.float8_e4m3fn if fp8 else kind).permute(order) for x in raw)
        pm.mla_gqa_rope_and_cache(q, k, v, pos, cs, 1, slots, torch.empty_like(q), kc, vc, err, scale, scale)
        o = torch.full((1, G * Hk, D), math.nan, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((1, G * Hk), math.nan, device=DEV)
        ws = pm.mla_gqa_decode(q[-1:], kc, vc, o, torch.tensor([0, ids.numel()], dtype=torch.int32, device=DEV),
                               ids, torch.tensor([(T - 1) % ps + 1], dtype=torch.int32, device=DEV), D ** -0.5,
                               scale, scale, lse)
        assert err.item() == 0 and pm.mla_check_error(ws) == 0
        assert not o.isnan().any()
        got.append([_bits(x.permute(order)) if x.dtype != torch.float32 else x for x in raw] + [o, lse])
    for a, b in zip(*got):
        assert torch.equal(a, b)

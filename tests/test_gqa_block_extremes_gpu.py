"""Decodes over block-scaled caches at the ends of what their inputs hold, on both kernels (up to 16
query rows a KV head and more)."""
import math

import pytest
import torch

from tests import gqa_block_ref as blk
from tests.test_gqa_block_gpu import DEV, Decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


@pytest.mark.parametrize("q", [-1e29, -3e31, -1e34, 1e33])
@pytest.mark.parametrize("rows,new", [(4, 1), (8, 4), (32, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_equal_scores_far_from_zero(pm, D, rows, new, q):
    """Every key is the same, so that all weights are, however far the scores are from zero: the mean of
    the values."""
    c = Decode([300, 5, 20001], [new] * 3, rows, 1, D, 16, 16)
    c.kc.view(torch.uint8).fill_(torch.tensor(1.0).to(blk.F8).view(torch.uint8).item())
    c.ks.fill_(1.0)
    c.vs.fill_(2.0 ** -6)
    c.q.fill_(q)
    o, lse, ws = c.run(pm, torch.float32)
    assert pm.mla_check_error(ws) == 0
    s = c.q[0, 0, 0].item() * D * c.sm
    at = 0
    for b, n in enumerate(c.pages.held):
        v = blk.values(c.pages, b, c.vc, c.vs).double()[:, 0]
        for t in range(new):
            seen = n - new + t + 1
            if seen > 0:
                # equal weights, exact in either kernel; fp32 sums of up to 20,001 values in pieces
                bound = 2.0 ** -20 * v[:seen].abs().mean(0) + 1e-30
                assert ((o[at + t].double() - v[:seen].mean(0)).abs() <= bound).all(), (b, t)
                # a score: fp32 products of a few factors, and ln's part far below its step
                assert ((lse[at + t].double() - s).abs() <= 2.0 ** -20 * abs(s)).all(), (b, t)
            else:
                assert (o[at + t] == 0).all() and torch.isneginf(lse[at + t]).all()
        at += new


def _scales(c, g, span, zero=None):
    """Scales of v over `span` powers of two and of k up to twice what they were, none a power of two;
    zero: positions of request 0 whose codes and scales are zero."""
    c.vs.copy_(torch.where(c.vs.isnan(), c.vs, torch.exp2(torch.rand(c.vs.shape, generator=g, device=DEV) * span - span / 2)))
    c.ks.copy_(torch.where(c.ks.isnan(), c.ks, c.ks * (1 + torch.rand(c.ks.shape, generator=g, device=DEV))))
    if zero:
        at = c.pages.where(0, *zero)
        for cache, scale in ((c.kc, c.ks), (c.vc, c.vs)):
            cache.view(torch.uint8)[at] = 0
            scale[at[0], at[1] // c.pages.bs] = 0


@pytest.mark.parametrize("span", [4, 20, 40])
@pytest.mark.parametrize("held,new,Hq,Hk,D,ps,bs,layout", [
    ([200, 1, 77], [1, 1, 1], 20, 1, 128, 16, 16, "nhd"),
    ([200, 31, 777], [4, 3, 4], 16, 2, 128, 64, 16, "hnd"),
    ([400, 31, 777], [4, 3, 4], 16, 2, 64, 16, 4, "nhd"),
    ([400, 64, 9001], [2, 1, 2], 36, 3, 64, 128, 128, "shared"),
    ([30001], [3], 8, 1, 128, 8, 1, "nhd"),
])
def test_decode_of_many_rows_and_scales_far_apart(pm, held, new, Hq, Hk, D, ps, bs, layout, span):
    """As test_decode_scales_far_apart, with more than 16 query rows a KV head."""
    c = Decode(held, new, Hq, Hk, D, ps, bs, layout)
    _scales(c, blk.gen(5, DEV), span, (128, 144))
    o, lse, ws = c.run(pm, torch.float32)
    assert pm.mla_check_error(ws) == 0
    c.check(o, lse, str(span), blk.LOST_MANY)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,new", [(4, 1), (3, 4), (20, 1), (8, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_into_outputs_with_strides(pm, D, rows, new, dtype):
    """Rows apart, heads outside tokens, slices of wider tensors: the same bits, and nothing beside them."""
    c = Decode([300, 0, 5, 9001], [new] * 4, 2 * rows, 2, D, 16, 16, pad=3)
    want, lse, ws = c.run(pm, dtype)
    n, (T, H, _) = 4 * new, c.q.shape
    for wide, view in ((torch.full((T, H, D + 3), 7.0, dtype=dtype, device=DEV), lambda x: x[:, :, :D]),
                       (torch.full((H, T + 1, D), 7.0, dtype=dtype, device=DEV), lambda x: x[:, 1:].transpose(0, 1)),
                       (torch.full((T, 3, H, D), 7.0, dtype=dtype, device=DEV), lambda x: x[:, 1])):
        o = view(wide)
        pm.mla_gqa_block_decode(c.q, c.kc, c.vc, c.ks, c.vs, o, c.qo, c.pages.indptr, c.pages.indices, c.pages.last,
                                new, c.sm, workspace=ws)
        assert pm.mla_check_error(ws) == 0
        assert torch.equal(o[:n], want[:n])
        o[:n] = 7.0
        assert (wide == 7.0).all()


@pytest.mark.parametrize("rows,new", [(4, 1), (8, 2), (32, 1), (8, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_infinite_scores(pm, D, rows, new):
    """A block of infinite key scale: rows that score it -inf give it no weight, +inf and NaN make theirs
    NaN; a row whose scores are all -inf is zero."""
    n, Hk = 300, 2
    c = Decode([n, 40], [new] * 2, rows * Hk, Hk, D, 16, 16)
    good, lse_good, ws = c.run(pm, torch.float32)
    page, slot = c.pages.where(0, 32, 48)
    code = torch.tensor(1.0).to(blk.F8).view(torch.uint8).item()
    c.kc.view(torch.uint8)[page, slot] = code
    c.ks[page[0], 0] = math.inf
    sign = torch.where(torch.arange(rows * Hk, device=DEV) % 3 == 0, 1.0, -1.0)        # of the heads' scores
    c.q.copy_((c.q.float().abs() * sign[:, None]).bfloat16())
    o, lse, _ = c.run(pm, torch.float32, ws=ws)
    up = sign > 0
    assert o[:new, up].isnan().all() and lse[:new, up].isnan().all()
    assert o[:new, ~up].isfinite().all() and lse[:new, ~up].isfinite().all()
    # the same without those positions: their keys out of reach by a finite score
    c.ks[page[0], 0] = 2.0 ** 40
    want, lse_want, _ = c.run(pm, torch.float32, ws=ws)
    assert torch.equal(o[:new, ~up], want[:new, ~up]) and torch.equal(lse[:new, ~up], lse_want[:new, ~up])
    assert torch.equal(o[new:], want[new:])
    # every score -inf
    page, slot = c.pages.where(0, 0, n)
    c.kc.view(torch.uint8)[page, slot] = code
    c.ks[page, slot // 16] = math.inf
    o, lse, _ = c.run(pm, torch.float32, ws=ws)
    assert (o[:new, ~up] == 0).all() and torch.isneginf(lse[:new, ~up]).all() and o[:new, up].isnan().all()
    assert torch.equal(o[new:], want[new:]) and pm.mla_check_error(ws) == 0

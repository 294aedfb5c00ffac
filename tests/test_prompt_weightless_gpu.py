"""Infinities and NaN among the values of keys without weight (scores of -inf, or too small for
fp32): 0 * inf is NaN in every row that sees such a key, on the causal edge and before it, in
whole and in cut units; a row whose keys all lack weight is zero."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _run(pm, q, k, v, keys, new):
    o = torch.full((q.shape[0], q.shape[1], v.shape[2]), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(o.shape[:2], math.nan, device=DEV)
    ptr = [torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (new, keys)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pm.mla_prompt_attention(q, k, v, o, *ptr, q.shape[2] ** -0.5, err, lse)
    assert err.item() == 0
    return o, lse


def _inputs(new, keys, D, DV):
    g = torch.Generator(device=DEV).manual_seed(keys + D)
    q = torch.randn(new, 4, D, generator=g, device=DEV).abs().add(0.1).bfloat16()     # positive
    k, v = (torch.randn(keys, 2, n, generator=g, device=DEV).bfloat16() for n in (D, DV))
    return q, k, v


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new,keys,at", [
    (300, 300, 3),          # an edge tile of the first queries', before the edge of the others'
    (300, 300, 170),
    (300, 300, 299),        # the last query's own key
    (150, 9000, 40),        # cut units: a tile that every query sees whole
    (150, 9000, 8900),      # the causal edge
])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("score", ["-inf", "small"])
def test_no_weight(pm, new, keys, at, D, DV, bad, score):
    q, k, v = _inputs(new, keys, D, DV)
    if score == "-inf":
        k[at, 1] = -math.inf
    else:
        # sums of D products below -0.1 * 2^11 / sqrt(D) D < -1600 against scores above -100:
        # exp of less than -1500 is zero in fp32
        k[at, 1] = -2.0 ** 11
    want, want_lse = _run(pm, q, k, v, keys, new)
    v[at, 1, 7] = bad
    o, lse = _run(pm, q, k, v, keys, new)
    rows = torch.arange(new, device=DEV) + keys - new >= at
    # a row that sees no other key: the weightless score is its only one
    alone = torch.arange(new, device=DEV) + keys - new == 0
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[rows & ~alone, 2:4, 7] = True
    assert o[hit].isnan().all()
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new,keys", [(300, 300), (70, 9000)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_rows_without_any_weight_are_zero(pm, new, keys, D, DV, bad):
    q, k, v = _inputs(new, keys, D, DV)
    k[:] = -math.inf
    v[::50] = bad
    v[-20:] = bad
    o, lse = _run(pm, q, k, v, keys, new)
    assert (o == 0).all() and lse.isneginf().all()


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new,keys,at", [(300, 300, 290), (300, 300, 3), (150, 9000, 8990)])
def test_weight_keeps_the_sign(pm, new, keys, at, D, DV):
    """A weighted infinity is an infinity; two of opposite signs are NaN; NaN is NaN."""
    q, k, v = _inputs(new, keys, D, DV)
    v[at, 0, 1] = math.inf
    v[at, 0, 2] = -math.inf
    v[at, 0, 3] = math.nan
    v[at, 0, 4], v[at + 1, 0, 4] = math.inf, -math.inf
    o, _ = _run(pm, q, k, v, keys, new)
    pos = torch.arange(new, device=DEV) + keys - new
    for h in (0, 1):
        assert (o[pos >= at, h, 1] == math.inf).all() and (o[pos >= at, h, 2] == -math.inf).all()
        assert o[pos >= at, h, 3].isnan().all()
        assert (o[pos == at, h, 4] == math.inf).all() and o[pos > at, h, 4].isnan().all()
    assert torch.isfinite(o[pos < at]).all() and torch.isfinite(o[:, 2:]).all()
    assert torch.isfinite(o[:, :, 0]).all() and torch.isfinite(o[:, :, 5:]).all()

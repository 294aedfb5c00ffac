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

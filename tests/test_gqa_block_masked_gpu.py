"""NaN among the newest positions: it reaches the rows that see it, in its own columns, and no other."""
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


CASES = [
    # held, new, Hq, Hk, D, ps, bs, layout
    ([5, 40, 33, 2, 700], [4, 4, 4, 2, 3], 4, 2, 128, 16, 16, "nhd"),
    ([5, 40, 33, 2, 700], [4, 4, 4, 2, 3], 3, 3, 64, 16, 8, "hnd"),
    ([130, 200, 65], [64, 1, 30], 3, 1, 64, 32, 32, "nhd"),
    ([5, 300, 40], [64, 64, 50], 2, 1, 128, 16, 16, "nhd"),            # queries that see nothing
    ([5, 300, 40, 129], [64, 64, 50, 2], 4, 4, 64, 8, 8, "nhd"),
    ([700, 3, 64], [3] * 3, 18, 3, 64, 8, 4, "nhd"),
    ([4100, 17, 127, 130], [5, 2, 5, 5], 48, 4, 128, 1024, 128, "hnd"),
    ([33001, 20], [4, 4], 16, 2, 128, 64, 64, "nhd"),
    ([33001, 20], [4, 4], 8, 2, 128, 4, 4, "nhd"),
    ([33001, 20], [2, 4], 10, 2, 64, 64, 64, "nhd"),
    ([300] * 200, [2] * 200, 20, 2, 64, 16, 16, "nhd"),
]


# 64-wide heads alone, and in pairs (which calls take whose page list has room for more than lies in L2)
@pytest.mark.parametrize("case,pairs", [(c, False) for c in CASES] + [(c, True) for c in CASES if c[4] == 64 and c[3] > 1])
def test_nan_reaches_the_rows_that_see_it(pm, case, pairs):
    held, new, Hq, Hk, D = case[:5]
    c = Decode(*case)
    if pairs:
        c.pages.indices = torch.cat([c.pages.indices, torch.full((1 << 22,), 1 << 30, dtype=torch.int32, device=DEV)])
    good, lse_good, ws = c.run(pm, torch.float32)
    g, head = Hq // Hk, Hk - 1
    most = max(blk.values(c.pages, b, c.vc, c.vs).abs().max().item() for b in range(len(held)) if held[b])
    ends = torch.tensor(new).cumsum(0).tolist()
    # (request, how many positions before the end, column): what is spoilt, one at a time and together
    spots = [(b, back, col) for b in (0, 1, len(held) - 1) for back, col in ((1, 0), (2, D - 1), (new[b], 37), (new[b] - 1, 17))
             if 1 <= back <= min(new[b], held[b])]
    for what in ("v code", "k code", "v scale", "k scale"):
        for group in [[s] for s in spots] + [spots]:
            want, lse_want = good.clone(), lse_good.clone()
            cache, scale = (c.vc, c.vs) if what[0] == "v" else (c.kc, c.ks)
            keep = cache.view(torch.uint8).clone(), scale.clone()
            for b, back, col in group:
                j, n, t = held[b] - back, held[b], new[b]
                page, slot = (x[0].item() for x in c.pages.where(b, j, j + 1))
                first = j
                if "code" in what:
                    cache.view(torch.uint8)[page, slot, head, col] = 0xFF if col % 2 else 0x7F
                else:
                    scale[page, slot // c.pages.bs, head] = math.nan
                    first = j // c.pages.bs * c.pages.bs
                for i in range(t):
                    if n - t + i >= first:
                        row = (ends[b] - t + i, slice(head * g, (head + 1) * g))
                        want[(*row, col) if what == "v code" else row] = math.nan
                        if what != "v code":
                            lse_want[row] = math.nan
            o, lse, _ = c.run(pm, torch.float32, ws=ws)
            cache.view(torch.uint8).copy_(keep[0])
            scale.copy_(keep[1])
            assert torch.equal(o.isnan(), want.isnan()), (what, group)
            assert torch.equal(lse.isnan(), lse_want.isnan()), (what, group)
            live, told = ~want.isnan(), ~lse_want.isnan()
            if g * max(new) <= 16:
                assert torch.equal(o[live], want[live]) and torch.equal(lse[told], lse_want[told]), (what, group)
            else:
                # rows of a head move their references together, so that others' bits may change with a
                # key: by the roundings of two results, weights' 2^-11 and up to 33,001 times 2^-25
                assert ((o[live] - want[live]).abs() <= 4 * 2.0 ** -10 * most).all(), (what, group)
                a, b = lse[told], lse_want[told]
                assert ((a == b) | ((a - b).abs() <= 2.0 ** -18 * (1 + b.abs()))).all(), (what, group)
    o, lse, _ = c.run(pm, torch.float32, ws=ws)
    assert torch.equal(o, good) and torch.equal(lse, lse_good) and pm.mla_check_error(ws) == 0

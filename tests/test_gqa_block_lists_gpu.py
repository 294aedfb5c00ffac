"""Lists with entries that make no sense: the requests that they belong to are left out, all others
are served."""
import random

import pytest
import torch

from tests import gqa_block_ref as blk
from tests.test_gqa_block_gpu import DEV, Append, _same

pytestmark = pytest.mark.gpu
FAR = (1000000, -1, 2 ** 31 - 1, -2 ** 31)


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _case(n, seed):
    rng = random.Random(seed)
    new = [rng.choice((0, 1, 3, 40, 64, 130) if n < 100 else (0, 1, 2, 5)) for _ in range(n)]
    return new, [rng.randrange(0, 90) for _ in range(n)]


@pytest.mark.parametrize("n,bad", [(3, {1: 1000000}), (3, {1: 10000}), (4, {0: -1}), (4, {4: 2 ** 31 - 1}), (4, {4: -2 ** 31})] +
                         [(n, {random.Random(7 * n + i).randrange(0, n + 1): FAR[(n + i) % 4] for i in range(k)})
                          for n, k in ((5, 1), (5, 2), (5, 5), (33, 1), (33, 5), (40, 2), (40, 5), (1100, 5))])
def test_append_serves_the_requests_beside_a_bad_token_list(pm, n, bad):
    new, before = _case(n, n) if n > 3 else ([64, 0, 64], [3, 0, 7])
    if n == 3 and 10000 in bad.values():
        new, before = [5, 5, 11], [0, 3, 40]
    case = (new, before, 4, 2, 64, 32, 1, 16, 16)
    a, old = Append(*case), Append(*case)
    kc, vc, ks, vs, q, k = a.want()
    starts = a.qo.tolist()
    for i, x in bad.items():
        a.qo[i] = x
    a.run(pm)
    assert a.err.item() == 2
    lost = [b for b in range(n) if b in bad or b + 1 in bad]
    total = sum(new)
    gone = torch.zeros(total, dtype=torch.bool, device=DEV)
    want = [x.view(torch.uint8).clone() if x.element_size() == 1 else x.clone() for x in (kc, vc, ks, vs)]
    for b in lost:
        gone[starts[b]:starts[b + 1]] = True
        page, slot = a.pages.where(b, 0, a.pages.held[b])
        for x, was in zip(want, (old.kc, old.vc, old.ks, old.vs)):
            at = (page, slot) if x.dtype == torch.uint8 else (page, slot // 16)
            x[at] = (was.view(torch.uint8) if x.dtype == torch.uint8 else was)[at]
    for x, got in zip(want, (a.kc, a.vc, a.ks, a.vs)):
        assert _same(got.view(blk.F8), x.view(blk.F8)) if x.dtype == torch.uint8 else _same(got, x)
    assert _same(a.k_out[:total][~gone], k[~gone]) and a.k_out[:total][gone].isnan().all()
    assert _same(a.q_out[:total], q)           # queries need no list but the end of the last one


@pytest.mark.parametrize("n,bad", [(3, {1: 1000000}), (4, {0: -1}), (4, {4: 2 ** 31 - 1}), (4, {4: -2 ** 31})] +
                         [(n, {random.Random(9 * n + i).randrange(0, n + 1): FAR[(n + i) % 4] for i in range(k)})
                          for n, k in ((5, 1), (5, 2), (33, 5), (700, 5), (1500, 1), (1500, 5))])
def test_gather_serves_the_requests_beside_a_bad_row_list(pm, n, bad):
    rng = random.Random(n)
    held = [rng.choice((0, 1, 3, 40, 70) if n < 100 else (0, 1, 2, 5)) for _ in range(n)]
    g = blk.gen(n, DEV)
    pages = blk.Pages(held, 16, 16, DEV)
    kc, vc, ks, vs = blk.caches(pages.pool, 16, 16, 2, 64, "nhd", DEV)
    blk.fill(pages, kc, ks, g)
    blk.fill(pages, vc, vs, g)
    rows = blk.sums(held, DEV)
    starts = rows.tolist()
    for i, x in bad.items():
        rows[i] = x
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k_rows, v_rows = (torch.full((sum(held) + 3, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pm.mla_gqa_block_gather(kc, vc, ks, vs, pages.indptr, pages.indices, pages.last, rows, k_rows, v_rows, err)
    assert err.item() == 2
    for got, cache, scale in ((k_rows, kc, ks), (v_rows, vc, vs)):
        want = torch.full_like(got, 7.0)
        for b in range(n):
            if held[b] and b not in bad and b + 1 not in bad:
                want[starts[b]:starts[b + 1]] = blk.values(pages, b, cache, scale).bfloat16()
        assert _same(got, want)

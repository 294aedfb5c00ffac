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

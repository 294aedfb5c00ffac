"""Page tables again: the pool's count in one word in and out."""
import random

import pytest
import torch

from tests.test_page_table_gpu import Step, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


@pytest.mark.parametrize("B", [5, 300, 3000])
def test_count_in_place_over_many_steps(pm, B):
    """Lists of many blocks, step after step on one pool without a wait between: as with the count
    in a word of its own, and no page handed out twice."""
    ps, width, steps = 2, 160 if B < 1000 else 40, 12
    rng = random.Random(B)
    seq, pool = [0] * B, B * width
    mine, other = (Step(seq, [0] * B, ps, width, pool=pool, n_idx=pool + 1, n_tok=0, seed=1) for _ in range(2))
    out = _ints([0])
    for _ in range(steps):
        new = [rng.randrange(0, 2 * ps * width // (2 * steps)) for _ in range(B)]
        seq = [n + t for n, t in zip(seq, new)]
        for s in (mine, other):
            s.seq_t, s.new_t = _ints(seq), _ints(new)
        for s, kw in ((mine, {}), (other, dict(count_out=out))):
            o = s.out
            pm.mla_build_page_table(s.seq_t, s.new_t, s.table, ps, o["qo"], o["key"], o["kv"], o["idx"], o["last"], s.err,
                                    free_pages=s.pages, free_count=s.count, free_count_out=kw.get("count_out", s.count))
        other.count.copy_(out)
    assert mine.err.tolist() == [0, 0] and other.err.tolist() == [0, 0]
    assert torch.equal(mine.count, other.count) and torch.equal(mine.table, other.table)
    assert torch.equal(mine.out["idx"], other.out["idx"])
    taken = mine.table[mine.table >= 0]
    assert taken.numel() == sum(-(-n // ps) for n in seq) == pool - mine.count.item()
    assert taken.unique().numel() == taken.numel()


def test_buffers_of_no_entries(pm):
    """Positions and slots of length 0 are lists like any other: cut, and flagged where the step has a
    token."""
    for t, bits in ((0, 0), (1, 8), (5, 8)):
        s = Step([7, 5], [0, t], 4, 2, n_tok=0)
        s.run(pm)
        assert s.err[0].item() == bits
        s.check()

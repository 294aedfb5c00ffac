"""Page tables built from request lengths, against plain lists."""
import random

import pytest
import torch

from tests import gqa_block_ref as blk

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("qo", "key", "kv", "idx", "last", "pos", "slots")


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Step:
    def __init__(self, seq, new, ps, width, pool=None, seed=0, n_idx=None, n_tok=None, stride=None):
        rng = random.Random(seed)
        self.seq, self.new, self.ps = seq, new, ps
        had = [max(0, min(width, -(-(n - t) // ps))) for n, t in zip(seq, new)]
        ids = rng.sample(range(2 * (sum(had) + (pool or 0)) + 50), sum(had) + (pool or 0))
        self.rows = []
        for n in had:
            self.rows.append([ids.pop() for _ in range(n)] + [-7] * (width - n))
        self.free = None if pool is None else list(ids)
        B = len(seq)
        wide = torch.full((B, stride or width), -7, dtype=torch.int32, device=DEV)
        self.table = wide[:, :width]
        if B and width:
            self.table.copy_(_ints(self.rows))
        pages = sum(-(-max(0, n) // ps) for n in seq)
        self.n_idx = pages + 3 if n_idx is None else n_idx
        self.n_tok = sum(max(0, t) for t in new) + 5 if n_tok is None else n_tok
        full = lambda n: torch.full((n,), -9, dtype=torch.int32, device=DEV)
        self.out = dict(qo=full(B + 1), key=full(B + 1), kv=full(B + 1), idx=full(self.n_idx), last=full(B),
                        pos=full(self.n_tok), slots=full(self.n_tok))
        self.err = torch.zeros(2, dtype=torch.int32, device=DEV)
        self.seq_t, self.new_t = _ints(seq), _ints(new)
        self.pages = None if pool is None else _ints(self.free)
        self.count = None if pool is None else _ints([len(self.free)])

    def run(self, pm, count_out=None, **kw):
        o = self.out
        pm.mla_build_page_table(self.seq_t, self.new_t, self.table, self.ps, o["qo"], o["key"], o["kv"], o["idx"],
                                o["last"], self.err, positions=o["pos"], slot_mapping=o["slots"],
                                free_pages=self.pages, free_count=self.count,
                                free_count_out=self.count if count_out is None else count_out, **kw)

    def check(self):
        want = blk.page_table(self.seq, self.new, self.rows, self.ps, self.free)
        live = min(len(want["idx"]), self.n_idx)
        want["idx"] = want["idx"][:live] + [-9] * (self.n_idx - live)
        n = min(len(want["pos"]), self.n_tok)
        want["pos"] = want["pos"][:n] + [0] * (self.n_tok - n)
        want["slots"] = want["slots"][:n] + [-1] * (self.n_tok - n)
        for name in NAMES:
            assert self.out[name].tolist() == want[name], name
        assert self.table.tolist() == self.rows
        if self.free is not None:
            assert self.count.item() == len(self.free)
        assert self.err[1].item() == 0


@pytest.mark.parametrize("pool", [None, 5000])
@pytest.mark.parametrize("seq,new,ps,width", [
    ([1], [1], 1, 1),
    ([1], [1], 16, 3),
    ([5, 0, 0, 33, 16, 17, 1], [1, 0, 0, 1, 1, 1, 1], 16, 4),
    ([130, 7, 300], [130, 0, 77], 64, 9),
    ([700, 0, 33, 4000], [700, 0, 2, 1], 1, 4001),
    ([1024, 1025, 2047], [1024, 1, 1023], 1024, 2),
    ([0, 0, 0], [0, 0, 0], 8, 0),
    ([], [], 8, 0),
    ([(i * 29) % 70 for i in range(300)], [(i * 29) % 70 // 2 for i in range(300)], 4, 20),
])
def test_tables(pm, seq, new, ps, width, pool):
    s = Step(seq, new, ps, width, pool, stride=width + 3)
    if pool is None:                     # every page is in the table already
        for b, n in enumerate(seq):
            for j in range(-(-n // ps)):
                s.rows[b][j] = 1000 + 50 * b + j
        if seq and width:
            s.table.copy_(_ints(s.rows))
    s.run(pm)
    assert s.err[0].item() == 0
    s.check()


@pytest.mark.parametrize("B", [1025, 5000, 16384])
def test_many_requests(pm, B):
    rng = random.Random(B)
    seq = [rng.randrange(0, 40) for _ in range(B)]
    new = [rng.randrange(0, n + 1) for n in seq]
    s = Step(seq, new, 8, 5, pool=5 * B)
    s.run(pm)
    assert s.err[0].item() == 0
    s.check()


def test_long_lists(pm):
    """One-token pages of 24 requests of 68,000 positions."""
    seq = [68000 - 7 * i for i in range(24)]
    s = Step(seq, [1] * 24, 1, 68000, pool=30)
    s.run(pm)
    assert s.err[0].item() == 0
    s.check()


def test_lengths_that_make_no_sense(pm):
    """Negative, more new than held, longer than the table: those requests count as empty."""
    s = Step([5, -1, 40, 9, 7, 33], [1, 0, 41, -2, 7, 1], 4, 8, pool=20)
    s.run(pm)
    assert s.err[0].item() == 2
    s.check()


def test_outputs_too_short(pm):
    s = Step([40, 33], [40, 1], 4, 12, pool=20, n_idx=7)
    s.run(pm)
    assert s.err[0].item() == 8
    s.check()
    s = Step([40, 33], [40, 1], 4, 12, pool=20, n_tok=9)
    s.run(pm)
    assert s.err[0].item() == 8
    s.check()


def test_pool_runs_out(pm):
    s = Step([40, 33, 9], [40, 33, 9], 4, 12, pool=13)
    s.run(pm)
    assert s.err[0].item() == 1 and s.count.item() == 0
    s.check()
    # a count that cannot be: no page is taken, the count stays
    for bad in (-1, 14):
        s = Step([8], [8], 4, 2, pool=13)
        s.count.fill_(bad)
        s.run(pm)
        assert s.err.tolist() == [1, 0] and s.count.item() == bad and s.table.tolist() == [[-1, -1]]
        assert s.out["slots"][:8].tolist() == [-1] * 8


def test_count_goes_to_another_tensor(pm):
    s = Step([40, 33, 9], [40, 33, 9], 4, 12, pool=40)
    out = _ints([-5])
    s.run(pm, count_out=out)
    assert s.count.item() == 40 and out.item() == 40 - 10 - 9 - 3


def test_no_positions(pm):
    s = Step([5, 6], [1, 1], 4, 3, pool=4)
    o = s.out
    pm.mla_build_page_table(s.seq_t, s.new_t, s.table, 4, o["qo"], o["key"], o["kv"], o["idx"], o["last"], s.err,
                            free_pages=s.pages, free_count=s.count, free_count_out=s.count)
    want = blk.page_table(s.seq, s.new, s.rows, 4, s.free)
    assert o["idx"][:4].tolist() == want["idx"] and s.table.tolist() == s.rows


def test_steps_in_a_graph(pm):
    """A captured step, replayed: lengths grow, pages are taken from the same stack as they go."""
    B, ps, width = 37, 4, 40
    s = Step([3 * i % 50 for i in range(B)], [0] * B, ps, width, pool=0)
    s.free = list(range(5000, 6000))
    s.pages, s.count = _ints(s.free), _ints([1000])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    s.n_idx = B * width
    s.out["idx"] = torch.full((s.n_idx,), -9, dtype=torch.int32, device=DEV)
    s.n_tok = B
    for name in ("pos", "slots"):
        s.out[name] = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    with torch.cuda.graph(graph, stream=side):
        s.run(pm)
    rng = random.Random(4)
    for _ in range(30):
        s.new = [rng.randrange(0, 2) for _ in range(B)]
        s.seq = [n + t for n, t in zip(s.seq, s.new)]
        s.seq_t.copy_(_ints(s.seq))
        s.new_t.copy_(_ints(s.new))
        s.out["idx"].fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert s.err[0].item() == 0
        s.check()

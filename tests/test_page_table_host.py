"""The page table's kernel on the host (CPU only): its own source runs as fibers, warps in any
order, so that what it reads and writes in place can be followed where a GPU would need luck."""
import ctypes
import os
import random
import re
import subprocess

import pytest

from tests import gqa_block_ref as blk

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_mla_latent_gb300", "csrc")
WARPS = 9


def _shared(m):
    """A block's shared array in the host's terms."""
    dynamic, kind, name, dim = m.groups()
    line = m.string.count("\n", 0, m.start())
    if dynamic:
        return f"{kind}* {name} = &sim::shared<{kind}>({line}, 1 << 20);"
    return f"auto& {name} = sim::shared<{kind}{dim or ''}>({line});"


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    def build(limit=None):
        d = tmp_path_factory.mktemp("page_table")
        text = open(os.path.join(CSRC, "mla_page_table.cu")).read().split('extern "C"')[0]
        text = re.sub(r"^#include.*$", "", text, flags=re.M)
        text = re.sub(r"(extern )?__shared__ (\w+) (\w+)(\[\w*\])?;", _shared, text)
        if limit is not None:
            text, n = re.subn(r"(kIntMax = )0x7FFFFFFF", rf"\g<1>{limit}", text)
            assert n == 1
        bits = re.search(r"enum : int \{[^}]*\};", open(os.path.join(CSRC, "ptx.cuh")).read()).group()
        (d / "page_table_kernel.inc").write_text("namespace pmla {\n" + bits + "\n}\n" + text)
        out = str(d / "libpagetable.so")
        r = subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{d}", "-o", out,
                            os.path.join(HERE, "native", "page_table_sim.cpp")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return ctypes.CDLL(out)
    return build


@pytest.fixture(scope="module")
def kernel(lib):
    return lib()


class Step:
    """A call's arrays, and what plain lists give for them."""

    def __init__(self, seq, new, ps, width, pool=None, blocks=1, n_idx=None, n_tok=None, table=None):
        ids = iter(range(100000, 900000, 7))
        self.seq, self.new, self.ps, self.width, self.blocks = seq, new, ps, width, blocks
        had = [min(width, max(0, -(-(n - t) // ps))) for n, t in zip(seq, new)]
        self.rows = table or [[next(ids) for _ in range(h)] + [-7] * (width - h) for h in had]
        self.free = None if pool is None else [next(ids) for _ in range(pool)]
        B = len(seq)
        pages = sum(-(-n // ps) for n in seq)
        self.n_idx = pages + 3 if n_idx is None else n_idx
        self.n_tok = sum(new) + 5 if n_tok is None else n_tok
        arr = lambda x: (ctypes.c_int32 * max(1, len(x)))(*x)
        full = lambda n: arr([-9] * n)
        self.a = dict(seq=arr(seq), new=arr(new), table=arr([x for r in self.rows for x in r]))
        self.a["free"] = None if pool is None else arr(self.free)
        self.a["count"] = self.a["count_out"] = None if pool is None else arr([pool])
        self.a.update(qo=full(B + 1), key=full(B + 1), kv=full(B + 1), idx=full(self.n_idx), last=full(B),
                      pos=full(self.n_tok), slots=full(self.n_tok), err=arr([0, 0]))

    def run(self, kernel, order=None):
        n = (ctypes.c_int64 * 7)(len(self.seq), self.width, self.ps.bit_length() - 1, len(self.free or []), self.n_idx,
                                 self.n_tok, self.blocks)
        ptr = (ctypes.c_void_p * 14)(*(None if x is None else ctypes.addressof(x) for x in self.a.values()))
        order = list(range(WARPS * self.blocks)) if order is None else order
        assert kernel.page_table(n, ptr, (ctypes.c_int * len(order))(*order)) == 0, "a wait without an end"

    def check(self, errors=0):
        rows, free = [list(r) for r in self.rows], None if self.free is None else list(self.free)
        want = blk.page_table(self.seq, self.new, rows, self.ps, free)
        want["idx"] += [-9] * (self.n_idx - len(want["idx"]))
        want["pos"] += [0] * (self.n_tok - len(want["pos"]))
        want["slots"] += [-1] * (self.n_tok - len(want["slots"]))
        for name in ("qo", "key", "kv", "last"):
            assert list(self.a[name])[:len(want[name])] == want[name], name
        for name, n in (("idx", self.n_idx), ("pos", self.n_tok), ("slots", self.n_tok)):
            assert list(self.a[name])[:n] == want[name][:n], name
        assert list(self.a["table"])[:len(rows) * self.width] == [x for r in rows for x in r]
        if free is not None:
            assert self.a["count"][0] == len(free)
        assert list(self.a["err"]) == [errors, 0]


ORDERS = [
    ("blocks in turn", lambda w, b: list(range(w * b))),
    ("blocks the other way", lambda w, b: [i * w + j for i in reversed(range(b)) for j in range(w)]),
    # each block's first warp, then block after block: the one whose first warp came last ends before
    # the others' later warps have begun
    ("first warps", lambda w, b: [i * w for i in range(b)] + [i * w + j for i in reversed(range(b)) for j in range(1, w)]),
    ("last warps first", lambda w, b: list(reversed(range(w * b)))),
] + [(f"shuffled {s}", lambda w, b, s=s: random.Random(s).sample(range(w * b), w * b)) for s in range(6)]


@pytest.mark.parametrize("name,order", ORDERS, ids=[n for n, _ in ORDERS])
def test_count_in_place_is_read_before_it_is_written(kernel, name, order):
    """The pool's count goes in and out in one word: no warp of any block may see the new one."""
    s = Step([40, 33, 9, 700], [40, 2, 9, 300], 4, 176, pool=120, blocks=3)
    s.run(kernel, order(WARPS, 3))
    s.check()
    # the same word once more
    t = Step([41, 34, 10, 701], [1] * 4, 4, 176, pool=7, blocks=3)
    t.run(kernel, order(WARPS, 3))
    t.check()


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("pool", [None, 3000])
@pytest.mark.parametrize("seq,new,ps,width", [
    ([], [], 8, 0), ([0, 0], [0, 0], 8, 0), ([1], [1], 1, 1), ([5, 0, 0, 33, 16, 17, 1], [1, 0, 0, 1, 1, 1, 1], 16, 4),
    ([700, 0, 33, 1300], [700, 0, 2, 1], 1, 1301),
    ([(i * 29) % 70 for i in range(300)], [(i * 29) % 70 // 2 for i in range(300)], 4, 20),
])
def test_tables(kernel, seq, new, ps, width, pool, blocks):
    table = None
    if pool is None:                       # every page is there already
        table = [[1000 + 50 * b + j for j in range(width)] for b in range(len(seq))]
    s = Step(seq, new, ps, width, pool, blocks, table=table)
    s.run(kernel)
    s.check()


@pytest.mark.parametrize("blocks", [1, 2])
def test_pages_past_the_largest_index(lib, blocks):
    """More pages in all than an index reaches (of 31 bits: here of 10, 999): bit 8, the sums end there,
    and no table entry, page or slot is given out."""
    s = Step([300, 500, 400, 7], [1, 100, 250, 7], 1, 500, pool=700, blocks=blocks, n_idx=900, n_tok=40)
    before = {n: list(s.a[n]) for n in ("table", "idx")}
    s.run(lib(limit=999))
    assert list(s.a["err"]) == [8, 0] and s.a["count"][0] == 700
    assert {n: list(s.a[n]) for n in before} == before
    assert list(s.a["kv"]) == list(s.a["key"]) == [0, 300, 800, 999, 999] and list(s.a["qo"]) == [0, 1, 101, 351, 358]
    assert list(s.a["pos"]) == [0] * 40 and list(s.a["slots"]) == [-1] * 40


@pytest.mark.parametrize("blocks", [1, 2])
def test_tokens_past_the_largest_index(lib, blocks):
    """More tokens than an index reaches, on fewer pages: those that the buffers hold are right."""
    s = Step([30, 1500], [20, 1400], 16, 100, pool=100, blocks=blocks, n_tok=900)
    s.run(lib(limit=999))
    want = blk.page_table(s.seq, s.new, s.rows, 16, s.free)
    # (slots are past the largest index here as well: -1, bit 1)
    assert list(s.a["err"]) == [9, 0] and s.a["count"][0] == len(s.free)
    assert list(s.a["pos"]) == want["pos"][:900] and list(s.a["slots"]) == [x if x <= 999 else -1 for x in want["slots"][:900]]
    assert list(s.a["idx"])[:len(want["idx"])] == want["idx"] and list(s.a["qo"]) == [0, 20, 999]

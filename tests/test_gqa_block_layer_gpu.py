"""The block-scaled operators together, as a serving loop runs them: the example's layer, and its
steps captured into a graph."""
import importlib.util
import math
import os

import pytest
import torch

from tests import gqa_block_ref as blk

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "grouped_head_layer", os.path.join(ROOT, "examples", "grouped_head_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_layer(example):
    # Keys and values are rounded to e4m3 once, by 2^-4 of each at most (a power-of-two scale and
    # its growth change normal codes exactly; below them the step is 2^-9 of the block's scale),
    # as in the layer with one scale: a value's own error, and five sigma of the weights'.
    assert example.run_blocks() <= 6 * (2.0 ** -4 + 5 * 0.036)


def test_layer_with_one_token_prompts(example):
    assert example.run_blocks(lens=(1, 1, 30), steps=6) <= 6 * (2.0 ** -4 + 5 * 0.036)


def _steps(pm, graph):
    """24 steps of 5 requests from nothing, tables, append and decode in one graph or call by call;
    everything the last step leaves."""
    B, hq, hk, d, ps, bs, pages = 5, 8, 2, 64, 16, 8, 64
    g = blk.gen(3, DEV)
    ints = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32, device=DEV)
    seq, new, table, idx = ints(B), ints(B, fill=1), ints(B, 8, fill=-1), ints(pages)
    free, count, err = torch.randperm(pages, generator=g, device=DEV).int(), ints(1, fill=pages), ints(2)
    qo, key, kv, last, pos, slots = ints(B + 1), ints(B + 1), ints(B + 1), ints(B), ints(B), ints(B)
    kc, vc = (torch.zeros(pages, ps, hk, d, dtype=torch.uint8, device=DEV).view(blk.F8) for _ in range(2))
    ks, vs = (torch.zeros(pages, ps // bs, hk, device=DEV) for _ in range(2))
    x = torch.randn(24, B, hq + 2 * hk, d, generator=g, device=DEV).bfloat16()
    q, k, v = (torch.empty(B, n, d, dtype=torch.bfloat16, device=DEV) for n in (hq, hk, hk))
    o, lse = torch.empty_like(q), torch.empty(B, hq, device=DEV)
    cs = blk.table(100, 64, DEV)
    ws = pm.make_gqa_block_decode_workspace(hq, hk, d, 1, DEV)

    def step():
        seq.add_(new)
        pm.mla_build_page_table(seq, new, table, ps, qo, key, kv, idx, last, err, positions=pos, slot_mapping=slots,
                                free_pages=free, free_count=count, free_count_out=count)
        pm.mla_gqa_block_append(q, k, v, pos, cs, 1, qo, kv, idx, last, q, kc, vc, ks, vs, err)
        pm.mla_gqa_block_decode(q, kc, vc, ks, vs, o, qo, kv, idx, last, 1, d ** -0.5, lse, ws)

    run = step
    if graph:
        side, captured = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(captured, stream=side):
            step()
        run = captured.replay
    outs = []
    for i in range(24):
        q.copy_(x[i, :, :hq])
        k.copy_(x[i, :, hq:hq + hk])
        v.copy_(x[i, :, hq + hk:])
        run()
        outs.append((o.clone(), lse.clone()))
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0] and pm.mla_check_error(ws) == 0
    assert seq.tolist() == [24] * B and count.item() == pages - 2 * B
    return outs + [(kc.view(torch.uint8), vc.view(torch.uint8)), (ks, vs), (table, idx)]


def test_steps_in_a_graph(pm):
    for a, b in zip(_steps(pm, False), _steps(pm, True)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_latent_decode_reads_the_built_tables(pm):
    """The tables of mla_build_page_table drive the latent cache's write and decode, too."""
    B, H, ps = 3, 12, 16
    g = blk.gen(9, DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    seq, new = ints([33, 1, 34]), ints([1, 1, 1])       # the first two take a page each
    table = ints([[7, 3, -1], [-1, -1, -1], [5, 2, 8]])
    out = {n: torch.zeros(m, dtype=torch.int32, device=DEV) for n, m in
           dict(qo=4, key=4, kv=4, idx=9, last=3, pos=3, slots=3).items()}
    err, count = ints([0, 0]), ints([2])
    pm.mla_build_page_table(seq, new, table, ps, out["qo"], out["key"], out["kv"], out["idx"], out["last"], err,
                            positions=out["pos"], slot_mapping=out["slots"], free_pages=ints([1, 9]),
                            free_count=count, free_count_out=count)
    assert out["kv"].tolist() == [0, 3, 4, 7] and count.item() == 0
    kv = torch.randint(0, 0x7E, (10, ps, 1, 576), generator=g, device=DEV, dtype=torch.uint8)
    q = torch.randint(0, 0x7E, (B, H, 576), generator=g, device=DEV, dtype=torch.uint8)
    one = torch.tensor(2.0 ** -8, device=DEV)
    o = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, H, device=DEV)
    ws = pm.mla_decode(q, kv, o, out["qo"], out["kv"], out["idx"], out["last"], 1, 576 ** -0.5, one, one, lse_out=lse)
    assert pm.mla_check_error(ws) == 0 and err.tolist() == [0, 0]
    val = lambda x: x.view(blk.F8).float().double() / 256
    for b in range(B):
        ids = out["idx"][out["kv"][b]:out["kv"][b + 1]].long()
        rows = val(kv[ids].flatten(0, 2))[:seq[b].item()]
        s = val(q[b]) @ rows.T * 576 ** -0.5
        want = torch.softmax(s, 1) @ rows[:, :512]
        # the decode's tolerance
        assert ((o[b].double() - want).abs() <= 1e-2 + 1e-2 * want.abs()).all()
        assert ((lse[b].double() - torch.logsumexp(s, 1)).abs() <= 1e-3).all()


def test_calls_on_another_stream(pm):
    """Each call runs on the stream that it is given, ordered by events alone."""
    from tests.test_gqa_block_gpu import Append, Decode
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        a = Append([30, 1, 200], [9, 100, 250], 4, 2, 128, 128, 1, 128, 64)
        want = a.want()
        c = Decode([300, 5000, 7], [2, 1, 3], 8, 2, 128, 16, 16)
        o0, lse0, _ = c.run(pm)
        side.wait_stream(torch.cuda.current_stream())
        a.run(pm, stream=stream)
        o, lse, ws = c.run(pm, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        a.check(want)
        assert torch.equal(o, o0) and torch.equal(lse, lse0)


def test_two_graphs_share_a_workspace(pm):
    """Decodes captured into two graphs with one workspace, replayed in turn."""
    from tests.test_gqa_block_gpu import Decode
    ws = pm.make_gqa_block_decode_workspace(16, 1, 128, 4, DEV)
    cases = [Decode([30001], [1], 8, 1, 128, 64, 64), Decode([20001, 40], [4, 2], 16, 1, 64, 16, 16)]
    graphs = []
    for c in cases:
        want = c.run(pm)[:2]
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            pm.mla_gqa_block_decode(c.q, c.kc, c.vc, c.ks, c.vs, o, c.qo, c.pages.indptr, c.pages.indices,
                                    c.pages.last, max(c.new), c.sm, lse, ws)
        graphs.append((graph, o, lse, want))
    for _ in range(3):
        for graph, o, lse, want in graphs:
            o.zero_()
            lse.zero_()
            graph.replay()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert pm.mla_check_error(ws) == 0


def test_caches_past_31_bits(pm):
    """Codes whose offsets pass 2^31 elements: the last pages of a 4.6 GB cache."""
    hk, d, ps, bs = 8, 128, 128, 64
    pages = 18000                               # 18,000 * 128 * 8 * 128 = 2.36e9 bytes each
    kc, vc = (torch.zeros(pages, ps, hk, d, dtype=torch.uint8, device=DEV).view(blk.F8) for _ in range(2))
    ks, vs = (torch.zeros(pages, ps // bs, hk, device=DEV) for _ in range(2))
    g = blk.gen(1, DEV)
    new = 200
    idx = torch.tensor([pages - 1, pages - 2, 0], dtype=torch.int32, device=DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    x = [torch.randn(new, n, d, generator=g, device=DEV).bfloat16() for n in (16, hk, hk)]
    err, q, k_out = ints([0, 0]), torch.empty_like(x[0]), torch.empty_like(x[1])
    lists = ints([0, 2]), idx, ints([new - ps])
    pm.mla_gqa_block_append(*x, torch.arange(new, dtype=torch.int32, device=DEV), blk.table(new, d, DEV), 1,
                            ints([0, new]), *lists, q, kc, vc, ks, vs, err, k_out=k_out)
    rows = torch.empty(2, new, hk, d, dtype=torch.bfloat16, device=DEV)
    pm.mla_gqa_block_gather(kc, vc, ks, vs, *lists, ints([0, new]), rows[0], rows[1], err)
    assert err[0].item() == 0
    for got, want in ((rows[0], k_out), (rows[1], x[2])):
        # one rounding to e4m3 (2^-4, below its normals half of 2^-9 of the scale, which is at most
        # 2^-7.8 of the block's largest) and two to bf16
        bound = want.float().abs() * (2.0 ** -4 + 2.0 ** -7) + 2.0 ** -10 * 2.0 ** -7.8 * want.float().abs().max()
        assert ((got.float() - want.float()).abs() <= bound).all()
    o, lse = torch.empty(1, 16, d, dtype=torch.float32, device=DEV), torch.empty(1, 16, device=DEV)
    ws = pm.mla_gqa_block_decode(q[-1:], kc, vc, ks, vs, o, ints([0, 1]), *lists, 1, d ** -0.5, lse)
    assert pm.mla_check_error(ws) == 0
    s = torch.einsum("hgd,nhd->hgn", q[-1].double().view(hk, 2, d), rows[0].double()) * d ** -0.5
    want = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), rows[1].double()).reshape(16, d)
    # weights rounded to 2^-11, against rows that are themselves rounded to bf16 exactly (powers of two)
    assert ((o[0].double() - want).abs() <= 2.0 ** -10 * rows[1].float().abs().max()).all()


def test_many_rows_past_31_bits(pm):
    """The same offsets for more than 16 rows a KV head, pairs of 64-wide heads among them."""
    ps, pages, held, new = 128, 18000, 300, 9
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    lists = ints([0, 3]), ints([pages - 1, 0, pages - 3]), ints([held - 2 * ps])
    g = blk.gen(2, DEV)
    both = [torch.zeros(pages * ps * 1024, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for hk, d in ((8, 128), (16, 64)):
        kc, vc = (x.view(pages, ps, hk, d) for x in both)
        ks, vs = (torch.zeros(pages, 2, hk, device=DEV) for _ in range(2))
        for cache, scale in ((kc, ks), (vc, vs)):
            for page in lists[1].tolist():
                x = torch.randn(ps, hk, d, generator=g, device=DEV) * 100
                cache[page] = x.clamp(-448, 448).to(blk.F8).view(torch.uint8)
                scale[page] = torch.exp2(torch.randint(-9, -5, (2, hk), generator=g, device=DEV).float())
        q = torch.randn(new, 2 * hk, d, generator=g, device=DEV).bfloat16()
        o, lse = torch.empty(q.shape, device=DEV), torch.empty(q.shape[:2], device=DEV)
        ws = pm.mla_gqa_block_decode(q, kc.view(blk.F8), vc.view(blk.F8), ks, vs, o, ints([0, new]), *lists, new,
                                     d ** -0.5, lse)
        assert pm.mla_check_error(ws) == 0
        j = torch.arange(held, device=DEV)
        page, slot = lists[1].long()[j // ps], j % ps
        k, v = (c.view(blk.F8)[page, slot].double() * s[page, slot // 64].double()[..., None] for c, s in ((kc, ks), (vc, vs)))
        s = torch.einsum("thgd,nhd->thgn", q.view(new, hk, 2, d).double(), k) * d ** -0.5
        s = s.masked_fill((j > held - new + torch.arange(new, device=DEV)[:, None])[:, None, None, :], -math.inf)
        want = torch.einsum("thgn,nhd->thgd", torch.softmax(s, -1), v).reshape(o.shape)
        # weights times scale rounded to 2^-11, or a multiple of 2^-24 of the largest; fp32 scores
        most = torch.einsum("thgn,nhd->thgd", torch.softmax(s, -1), v.abs()).reshape(o.shape)
        assert ((o.double() - want).abs() <= 2.0 ** -9 * most + 2.0 ** -24 * held * v.abs().max()).all()


def test_decodes_of_few_and_many_rows_share_a_workspace(pm):
    """In turn on one workspace, the one-scale decode among them; too small and scattered ones are
    refused."""
    from tests.test_gqa_block_gpu import Decode
    ws = max((pm.make_gqa_block_decode_workspace(32, 2, d, 4, DEV) for d in (64, 128)), key=lambda x: x.numel())
    cases = [Decode([30001, 5], [1, 1], 32, 2, 128, 64, 64), Decode([20001, 40], [4, 2], 16, 2, 128, 16, 16),
             Decode([30001], [4], 32, 2, 64, 64, 64)]
    want = [c.run(pm)[:2] for c in cases]
    one = torch.tensor(0.02, device=DEV)
    c = cases[0]
    plain = torch.empty_like(c.q)
    for i in range(3):
        for c, (o0, lse0) in zip(cases, want):
            o, lse, _ = c.run(pm, ws=ws)
            assert torch.equal(o, o0) and torch.equal(lse, lse0)
        c = cases[0]
        pm.mla_gqa_decode(c.q, c.kc, c.vc, plain, c.pages.indptr, c.pages.indices, c.pages.last, c.sm, one, one,
                          workspace=ws)
        if i == 0:
            first = plain.clone()
        assert torch.equal(plain, first)
    assert pm.mla_check_error(ws) == 0
    with pytest.raises(ValueError):
        cases[1].run(pm, ws=torch.zeros(1, dtype=torch.uint8, device=DEV).expand(1 << 26))
    with pytest.raises(pm.MlaError):
        cases[1].run(pm, ws=ws[:4096])

"""Causal attention of packed prompts, against fp64."""
import math

import pytest
import torch

from tests import gqa_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _case(new, keys, Hq, Hk, D, DV, seed=0, strided=False, std=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed + sum(new) + 3 * sum(keys) + D)
    T, L = sum(new), sum(keys)

    def rand(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * s).bfloat16()

    if strided:
        # views of wider rows; keys and values of one tensor
        q = rand(T, Hq, D + 24, s=std)[:, :, 8:D + 8]
        kv = rand(L, Hk, D + DV + 8)
        k, v = kv[:, :, :D], kv[:, :, D:D + DV]
        o = torch.full((T, Hq, DV + 16), math.nan, dtype=torch.bfloat16, device=DEV)[:, :, :DV]
    else:
        q, k, v = rand(T, Hq, D, s=std), rand(L, Hk, D), rand(L, Hk, DV)
        o = torch.full((T, Hq, DV), math.nan, dtype=torch.bfloat16, device=DEV)

    def ptr(x):
        out = [0]
        for n in x:
            out.append(out[-1] + n)
        return torch.tensor(out, dtype=torch.int32, device=DEV)

    return dict(q=q, k=k, v=v, o=o, lse=torch.full((T, Hq), math.nan, device=DEV), qo=ptr(new), kv=ptr(keys),
                sm=D ** -0.5, err=torch.zeros(1, dtype=torch.int32, device=DEV), new=new, keys=keys)


def _run(pm, c):
    pm.mla_prompt_attention(c["q"], c["k"], c["v"], c["o"], c["qo"], c["kv"], c["sm"], c["err"], c["lse"])


def _check(c, what, rows=None):
    """Every request (or `rows` evenly spaced query tokens of each) against fp64."""
    Hq, Hk = c["q"].shape[1], c["k"].shape[1]
    G, D = Hq // Hk, c["q"].shape[2]
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(c["new"], c["keys"])):
        t = torch.arange(n, device=DEV)
        if rows and n > rows:
            t = torch.cat([t[:2], t[torch.linspace(0, n - 1, rows, device=DEV).long()], t[-2:]])
        for h in range(Hq if n else 0):
            k = c["k"][k0:k0 + m, h // G].double()
            v = c["v"][k0:k0 + m, h // G].double()
            out = ref.attend(c["q"][q0 + t, h].double(), k, v, c["sm"], m - n + t + 1)
            ref.check(c["o"][q0 + t, h], c["lse"][q0 + t, h], out, max(m, 1), D, ref.BF16, ref.BF16,
                      f"{what}: request {b} ({n} of {m}), head {h}")
        q0, k0 = q0 + n, k0 + m


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new,keys,Hq,Hk,strided", [
    ([1], [1], 1, 1, False),
    ([1, 2, 3], [1, 2, 3], 4, 2, False),
    ([127, 128, 129], None, 2, 2, True),
    ([255, 256, 257], None, 1, 1, False),
    ([33, 0, 64, 65, 0], None, 8, 2, False),
    ([200], None, 7, 1, True),                     # groups that do not divide a tile
    ([61, 300], None, 12, 1, False),
    ([40], None, 128, 1, False),                   # a token a tile
    ([9, 5], None, 100, 1, False),
    ([5, 1, 100], [300, 129, 1000], 4, 2, True),   # prefixes
    ([1, 1, 1, 1], [0, 128, 640, 641], 3, 1, False),
    ([300, 10, 5], [290, 0, 1], 2, 1, False),      # queries that see nothing
    ([700], [1400], 6, 2, False),
])
def test_prompt(pm, new, keys, Hq, Hk, strided, D, DV):
    c = _case(new, keys or new, Hq, Hk, D, DV, strided=strided)
    _run(pm, c)
    assert c["err"].item() == 0
    _check(c, f"{D}/{DV}")
    first, lse = c["o"].clone(), c["lse"].clone()
    _run(pm, c)
    assert torch.equal(first, c["o"]) and torch.equal(lse, c["lse"])


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
def test_prompt_long(pm, D, DV):
    """Many K/V tiles (the ring wraps at every chunk), many CTAs."""
    c = _case([2500, 31, 4096], [2500, 8031, 4100], 8, 2, D, DV)
    _run(pm, c)
    assert c["err"].item() == 0
    _check(c, "long", rows=300)


def test_prompt_many_requests(pm):
    new = [(i * 29) % 70 for i in range(150)]
    keys = [n + (i * 13) % 200 for i, n in enumerate(new)]
    c = _case(new, keys, 4, 2, 64, 64)
    _run(pm, c)
    assert c["err"].item() == 0
    _check(c, "150 requests")


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
def test_prompt_growing_scores(pm, D, DV):
    """Scores that keep growing along the keys, so that the maximum is raised again and
    again, and ones that fall."""
    for sign in (1.0, -1.0):
        c = _case([600], [1500], 2, 1, D, DV)
        ramp = torch.linspace(0, 6, 1500, device=DEV)[:, None, None] * sign
        u = torch.randn(D, device=DEV)
        c["k"] += (ramp * u).bfloat16()
        c["q"] += u.bfloat16()
        _run(pm, c)
        _check(c, f"sign {sign}", rows=150)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
def test_prompt_non_finite_values(pm, D, DV, bad):
    """Non-finite keys and values reach the rows that see them and no others: neither earlier
    queries of the request nor the requests beside it."""
    new, keys = [150, 200, 90], [150, 350, 90]
    clean = _case(new, keys, 4, 2, D, DV)
    _run(pm, clean)
    c = _case(new, keys, 4, 2, D, DV)
    at = 150 + 150 + 77                       # request 1's query 77, seen by its queries 77 ..
    c["v"][at, 1, 5] = bad
    _run(pm, c)
    o, want = c["o"], clean["o"]
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[150 + 77:350, 2:4, 5] = True
    assert torch.equal(o[~hit], want[~hit])
    got = o[hit]
    assert (got.isnan() if math.isnan(bad) else got == math.inf).all()
    # a key: every column of the rows that see it
    c = _case(new, keys, 4, 2, D, DV)
    c["k"][at, 0, 3] = math.nan
    _run(pm, c)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[150 + 77:350, 0:2] = True
    assert torch.equal(c["o"][~hit], want[~hit]) and c["o"][hit].isnan().all()
    # an early value: every query of the request
    c = _case(new, keys, 4, 2, D, DV)
    c["v"][150 + 3, 0, 0] = bad
    _run(pm, c)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[150:350, 0:2, 0] = True
    assert torch.equal(c["o"][~hit], want[~hit])
    assert (~torch.isfinite(c["o"][hit])).all()


def test_prompt_keys_at_minus_infinity(pm):
    """A key whose scores are -inf has no weight; a query of nothing else gives zero."""
    c = _case([130], [130], 2, 1, 64, 64)
    c["q"].abs_()
    want = _case([130], [130], 2, 1, 64, 64)
    c["k"][0] = -math.inf
    _run(pm, c)
    assert (c["o"][0] == 0).all() and c["lse"][0].isneginf().all()
    assert torch.isfinite(c["o"]).all() and torch.isfinite(c["lse"][1:]).all()
    q, k, v = c["q"].double(), want["k"].double(), want["v"].double()
    for t in (1, 64, 129):
        out = ref.attend(q[t:t + 1, 0], k[1:t + 1, 0], v[1:t + 1, 0], c["sm"], torch.tensor([t], device=DEV))
        ref.check(c["o"][t:t + 1, 0], c["lse"][t:t + 1, 0], out, t, 64, ref.BF16, ref.BF16, f"query {t}")


def test_prompt_bad_ranges(pm):
    good = _case([50, 60, 70], [50, 60, 70], 4, 2, 64, 64)
    _run(pm, good)
    c = _case([50, 60, 70], [50, 60, 70], 4, 2, 64, 64)
    c["kv"][3] = 10 ** 6                      # leaves the keys: request 2 has none
    _run(pm, c)
    assert c["err"].item() == 2
    assert torch.equal(c["o"][:110], good["o"][:110]) and (c["o"][110:] == 0).all()
    assert c["lse"][110:].isneginf().all()
    c = _case([50, 60, 70], [50, 60, 70], 4, 2, 64, 64)
    c["qo"][1] = 10 ** 6                      # requests 0 and 1 are left out
    _run(pm, c)
    assert c["err"].item() == 2
    assert torch.equal(c["o"][110:], good["o"][110:]) and c["o"][:110].isnan().all()
    c = _case([50, 60], [50, 60], 4, 2, 64, 64)
    c["qo"][2] = 80                           # rows of no request stay as they were
    c["new"] = [50, 30]
    _run(pm, c)
    assert c["err"].item() == 0 and c["o"][80:].isnan().all() and not c["o"][:80].isnan().any()


@pytest.mark.parametrize("keys", [[300, 500], [9000, 2500]])       # whole; cut and joined
def test_prompt_in_a_graph(pm, keys):
    c = _case([300, 20], keys, 8, 2, 128, 128)
    _run(pm, c)
    want = c["o"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(pm, c)
    for _ in range(3):
        c["o"].fill_(math.nan)
        graph.replay()
        assert torch.equal(c["o"], want)


def test_prompt_scales(pm):
    for sm in (1e-30, 1e-3, 3.0):
        c = _case([200, 70], [200, 1100], 4, 2, 128, 128)
        c["sm"] = sm
        _run(pm, c)
        _check(c, f"sm_scale {sm}")


def test_prompt_back_to_back(pm):
    """Calls of different shapes on one workspace, one behind the other: a call's first kernel
    does not run into the join before it."""
    cases = [_case([40], [30000 + 700 * i], 8, 2, 128, 128, seed=i) for i in range(4)]
    alone = []
    for c in cases:
        _run(pm, c)
        alone.append(c["o"].clone())
        torch.cuda.synchronize()
    ws = torch.empty(pm.mla_get_prompt_workspace_size(40000, 128), dtype=torch.uint8, device=DEV)
    for _ in range(5):
        for c in cases:
            c["o"].fill_(math.nan)
        for c in cases:
            pm.mla_prompt_attention(c["q"], c["k"], c["v"], c["o"], c["qo"], c["kv"], c["sm"], c["err"],
                                    c["lse"], workspace=ws)
        for c, want in zip(cases, alone):
            assert torch.equal(c["o"], want)


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new,keys,Hq,Hk", [
    ([16], [40000], 4, 2),                         # few rows over many keys: cut many times
    ([1, 300, 700], [5000, 9000, 700], 6, 2),
    ([2100, 5, 2100], [2100, 2049, 4200], 2, 1),
])
def test_prompt_cut_between_sms(pm, new, keys, Hq, Hk, D, DV):
    """With a workspace long units are cut between SMs and joined; without one they are not.
    Both are right, each gives the same bits again."""
    c = _case(new, keys, Hq, Hk, D, DV)
    _run(pm, c)
    assert c["err"].item() == 0
    _check(c, "cut", rows=100)
    first, lse = c["o"].clone(), c["lse"].clone()
    n = pm.mla_get_prompt_workspace_size(sum(keys), DV)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)       # stale NaN
    pm.mla_prompt_attention(c["q"], c["k"], c["v"], c["o"], c["qo"], c["kv"], c["sm"], c["err"], c["lse"],
                            workspace=ws)
    assert torch.equal(first, c["o"]) and torch.equal(lse, c["lse"])
    with pytest.raises(pm.MlaError):
        pm.mla_prompt_attention(c["q"], c["k"], c["v"], c["o"], c["qo"], c["kv"], c["sm"], c["err"],
                                workspace=ws[:n // 2])
    c["o"].fill_(math.nan)
    d = [pm._packed(c[x], 0) for x in ("q", "k", "v", "o", "qo", "kv")]
    assert pm._lib.mla_prompt_attention(*d, c["sm"], pm._packed(c["lse"], 0), c["err"].data_ptr(), None, 0,
                                        torch.cuda.current_stream().cuda_stream) == 0
    _check(c, "whole", rows=100)


def test_prompt_non_finite_values_in_cut_units(pm):
    new, keys = [40, 30], [6000, 7000]
    clean = _case(new, keys, 2, 1, 128, 128)
    _run(pm, clean)
    for at, rows in ((100, range(0, 40)), (6000 - 40 + 7, range(7, 40)), (6000 + 6990, range(60, 70))):
        c = _case(new, keys, 2, 1, 128, 128)
        c["v"][at, 0, 9] = math.inf
        _run(pm, c)
        hit = torch.zeros_like(c["o"], dtype=torch.bool)
        hit[list(rows), :, 9] = True
        assert torch.equal(c["o"][~hit], clean["o"][~hit])
        assert (~torch.isfinite(c["o"][hit])).all()


def test_prompt_on_another_stream(pm):
    c = _case([500, 20], [5000, 500], 8, 2, 128, 128)
    _run(pm, c)
    want = c["o"].clone()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        c["o"].fill_(math.nan)
        torch.cuda.synchronize()
        pm.mla_prompt_attention(c["q"], c["k"], c["v"], c["o"], c["qo"], c["kv"], c["sm"], c["err"], c["lse"],
                                stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(c["o"], want)

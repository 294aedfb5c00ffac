"""Prompt attention called again, each time into outputs that hold nothing of the call before."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _indptr(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new,keys,Hq,Hk", [
    ([61, 300, 0, 7], [61, 300, 0, 400], 12, 3),   # whole units
    ([300, 10, 5], [290, 0, 1], 2, 1),             # queries that see nothing
    ([16], [40000], 4, 2),                         # cut many times
    ([2100, 5, 2100], [2100, 2049, 4200], 2, 1),
])
def test_same_bits_again(pm, new, keys, Hq, Hk, D, DV):
    g = torch.Generator(device=DEV).manual_seed(sum(keys))
    T, L = sum(new), sum(keys)
    q = (torch.randn(T, Hq, D, generator=g, device=DEV) * 1.5).bfloat16()
    k, v = (torch.randn(L, Hk, n, generator=g, device=DEV).bfloat16() for n in (D, DV))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = pm.mla_get_prompt_workspace_size(L, DV)
    first = None
    for workspace in (None, None, "stale", "stale"):
        o = torch.full((T, Hq, DV), math.nan, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((T, Hq), math.nan, device=DEV)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if workspace and n else None
        pm.mla_prompt_attention(q, k, v, o, _indptr(new), _indptr(keys), D ** -0.5, err, lse, workspace=ws)
        assert not o.isnan().any() and not lse.isnan().any()
        if first is None:
            first = o, lse
        assert torch.equal(first[0], o) and torch.equal(first[1], lse)
    assert err.item() == 0

"""Outputs that are lazy clones of other tensors: what is written is theirs alone."""
import pytest
import torch

from tests.test_gqa_block_gpu import Append, Decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def test_outputs_that_are_lazy_clones(pm):
    a = Append([30, 1], [9, 100], 4, 2, 128, 128, 1, 128, 64)
    want = a.want()
    first = torch.zeros(31, 4, 128, dtype=torch.bfloat16, device="cuda")
    a.q_out = first._lazy_clone()
    a.run(pm)
    a.check(want)
    assert (first == 0).all()
    c = Decode([300, 7], [1, 1], 8, 2, 128, 16, 16)
    o, lse, ws = c.run(pm)
    first = torch.zeros_like(o)
    clone = first._lazy_clone()
    pm.mla_gqa_block_decode(c.q, c.kc, c.vc, c.ks, c.vs, clone, c.qo, c.pages.indptr, c.pages.indices, c.pages.last, 1,
                            c.sm, workspace=ws)
    assert torch.equal(clone, o) and (first == 0).all()

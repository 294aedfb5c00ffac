"""Outputs whose rows share memory are refused by the grouped-head entry points, before anything
is enqueued (CPU only).  Calls that pass the checks of strides end at a head width that no kernel
has, so that nothing is launched on a machine with a GPU either."""
import pytest

from tests.test_gqa_abi import (BF, F32, I32, INVALID, UNSUPPORTED, _append, _append_args, _decode,
                                _decode_args, _prompt, _prompt_args, _t)

D = 96


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _calls(pm, tokens=4):
    """{name: (call, arguments, the outputs' names and heads)} at a width without a kernel."""
    T = tokens
    a = _append_args(pm)
    for key, n, heads in (("q", 0, 8), ("k", 1, 2), ("v", 2, 2), ("qo", 6, 8), ("ko", 7, 2)):
        a[key] = _t(pm, n, BF, [T, heads, D])
    a.update(pos=_t(pm, 3, I32, [T]), cs=_t(pm, 4, F32, [64, D]), slots=_t(pm, 5, I32, [T]))
    a["kc"], a["vc"] = (_t(pm, n, BF, [10, 16, 2, D]) for n in (8, 9))
    d = _decode_args(pm)
    d.update(q=_t(pm, 0, BF, [T, 8, D]), kc=_t(pm, 1, BF, [10, 16, 2, D]), vc=_t(pm, 2, BF, [10, 16, 2, D]),
             o=_t(pm, 3, BF, [T, 8, D]), ptr=_t(pm, 4, I32, [T + 1]), last=_t(pm, 6, I32, [T]), lse=None)
    p = _prompt_args(pm)
    p.update(q=_t(pm, 0, BF, [T, 8, D]), k=_t(pm, 1, BF, [9, 2, D]), v=_t(pm, 2, BF, [9, 2, D]),
             o=_t(pm, 3, BF, [T, 8, D]), lse=None)
    return {"append": (_append, a, (("qo", 8), ("ko", 2))), "decode": (_decode, d, (("o", 8),)),
            "prompt": (_prompt, p, (("o", 8),))}


@pytest.mark.parametrize("name", ["append", "decode", "prompt"])
@pytest.mark.parametrize("strides", [
    lambda T, H: [0, D, 1],                  # every token's row in one place
    lambda T, H: [H * D, 0, 1],              # every head's
    lambda T, H: [H * D, D - 8, 1],          # heads that overlap
    lambda T, H: [H * D - 8, D, 1],          # a token's last head and the next one's first
    lambda T, H: [D, D, 1],
    lambda T, H: [D, T * D - 8, 1],
])
def test_overlapping_outputs_are_refused(pm, name, strides):
    call, args, outs = _calls(pm)[name]
    for key, heads in outs:
        out = _t(pm, 12, BF, [4, heads, D], strides(4, heads))
        assert call(pm, {**args, key: out}) == INVALID, key


def test_overlapping_fp32_outputs_are_refused(pm):
    call, args, _ = _calls(pm)["decode"]
    assert call(pm, {**args, "o": _t(pm, 12, F32, [4, 8, D], [8 * D, D - 1, 1])}) == INVALID
    assert call(pm, {**args, "o": _t(pm, 12, F32, [4, 8, D], [8 * (D + 1), D + 1, 1])}) == UNSUPPORTED


@pytest.mark.parametrize("name", ["append", "decode", "prompt"])
@pytest.mark.parametrize("strides", [
    lambda T, H: [H * D, D, 1],
    lambda T, H: [H * D + 8, D, 1],          # wider rows
    lambda T, H: [2 * H * D, 2 * D, 1],
    lambda T, H: [D, T * D, 1],              # heads outside tokens
])
def test_outputs_apart_are_taken(pm, name, strides):
    call, args, outs = _calls(pm)[name]
    assert call(pm, args) == UNSUPPORTED
    for key, heads in outs:
        out = _t(pm, 12, BF, [4, heads, D], strides(4, heads))
        assert call(pm, {**args, key: out}) == UNSUPPORTED, key


@pytest.mark.parametrize("name", ["append", "decode", "prompt"])
def test_a_single_row_has_nothing_to_overlap(pm, name):
    call, args, outs = _calls(pm, tokens=1)[name]
    for key, heads in outs:
        for first in (0, 8):                 # the stride of one token is never stepped
            out = _t(pm, 12, BF, [1, heads, D], [first, D, 1])
            assert call(pm, {**args, key: out}) == UNSUPPORTED, key

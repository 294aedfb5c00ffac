"""Host-side refusals of the grouped-head entry points (CPU only: nothing is enqueued)."""
import ctypes

import pytest

F8, BF, F32, I32 = 1, 2, 3, 4
INVALID, UNSUPPORTED, SMALL = 1, 2, 3
BASE = 1 << 40


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _t(pm, n, dtype, shape, stride=None, ptr=None):
    d = pm.MlaTensor()
    d.ptr = BASE + (n << 28) if ptr is None else (ptr or None)
    d.ndim, d.dtype = len(shape), dtype
    if stride is None:
        stride, acc = [], 1
        for s in reversed(shape):
            stride.insert(0, acc)
            acc *= s
    for i, (s, st) in enumerate(zip(shape, stride)):
        d.shape[i], d.stride[i] = s, st
    return d


def _r(d):
    return ctypes.byref(d) if d is not None else None


def _append_args(pm):
    T, Hq, Hk, D = 4, 8, 2, 128
    return dict(q=_t(pm, 0, BF, [T, Hq, D]), k=_t(pm, 1, BF, [T, Hk, D]), v=_t(pm, 2, BF, [T, Hk, D]),
                pos=_t(pm, 3, I32, [T]), cs=_t(pm, 4, F32, [64, 128]), neox=1, slots=_t(pm, 5, I32, [T]),
                ks=None, vs=None, qo=_t(pm, 6, BF, [T, Hq, D]), ko=_t(pm, 7, BF, [T, Hk, D]),
                kc=_t(pm, 8, BF, [10, 16, Hk, D]), vc=_t(pm, 9, BF, [10, 16, Hk, D]),
                err=BASE + (10 << 28))


def _append(pm, a):
    return pm._lib.mla_gqa_rope_and_cache(
        _r(a["q"]), _r(a["k"]), _r(a["v"]), _r(a["pos"]), _r(a["cs"]), a["neox"], _r(a["slots"]),
        _r(a["ks"]), _r(a["vs"]), _r(a["qo"]), _r(a["ko"]), _r(a["kc"]), _r(a["vc"]),
        ctypes.c_void_p(a["err"]), None)


def _fp8_caches(pm, **kw):
    return dict(kc=_t(pm, 8, F8, [10, 16, 2, 128]), vc=_t(pm, 9, F8, [10, 16, 2, 128]),
                ks=_t(pm, 11, F32, []), vs=_t(pm, 12, F32, [1]), **kw)


@pytest.mark.parametrize("name,change,status", [
    ("q type", lambda pm: dict(q=_t(pm, 0, F32, [4, 8, 128])), INVALID),
    ("q rank", lambda pm: dict(q=_t(pm, 0, BF, [4, 1024])), INVALID),
    ("q missing", lambda pm: dict(q=None), INVALID),
    ("q base", lambda pm: dict(q=_t(pm, 0, BF, [4, 8, 128], ptr=BASE + 8)), INVALID),
    ("q stride", lambda pm: dict(q=_t(pm, 0, BF, [4, 8, 128], [1028, 128, 1])), INVALID),
    ("q columns apart", lambda pm: dict(q=_t(pm, 0, BF, [4, 8, 128], [2048, 256, 2])), INVALID),
    ("heads not grouped", lambda pm: dict(k=_t(pm, 1, BF, [4, 3, 128])), INVALID),
    ("v width", lambda pm: dict(v=_t(pm, 2, BF, [4, 2, 64])), INVALID),
    ("k tokens", lambda pm: dict(k=_t(pm, 1, BF, [5, 2, 128])), INVALID),
    ("positions length", lambda pm: dict(pos=_t(pm, 3, I32, [3])), INVALID),
    ("slots type", lambda pm: dict(slots=_t(pm, 5, F32, [4])), INVALID),
    ("table width", lambda pm: dict(cs=_t(pm, 4, F32, [64, 24])), INVALID),
    ("table too wide", lambda pm: dict(cs=_t(pm, 4, F32, [64, 144])), INVALID),
    ("table stride", lambda pm: dict(cs=_t(pm, 4, F32, [64, 128], [130, 1])), INVALID),
    ("neox", lambda pm: dict(neox=2), INVALID),
    ("q_out shape", lambda pm: dict(qo=_t(pm, 6, BF, [4, 7, 128])), INVALID),
    ("k_out shape", lambda pm: dict(ko=_t(pm, 7, BF, [4, 8, 128])), INVALID),
    ("cache heads", lambda pm: dict(kc=_t(pm, 8, BF, [10, 16, 4, 128])), INVALID),
    ("cache types differ", lambda pm: dict(vc=_t(pm, 9, F8, [10, 16, 2, 128])), INVALID),
    ("cache strides differ", lambda pm: dict(vc=_t(pm, 9, BF, [10, 16, 2, 128], [4096, 128, 2048, 1])), INVALID),
    ("slots overlap", lambda pm: dict(kc=_t(pm, 8, BF, [10, 16, 2, 128], [4096, 128, 128, 1]),
                                      vc=_t(pm, 9, BF, [10, 16, 2, 128], [4096, 128, 128, 1])), INVALID),
    ("page size", lambda pm: dict(kc=_t(pm, 8, BF, [10, 24, 2, 128]),
                                  vc=_t(pm, 9, BF, [10, 24, 2, 128])), UNSUPPORTED),
    ("page too large", lambda pm: dict(kc=_t(pm, 8, BF, [10, 2048, 2, 128]),
                                       vc=_t(pm, 9, BF, [10, 2048, 2, 128])), UNSUPPORTED),
    ("slots past 31 bits", lambda pm: dict(kc=_t(pm, 8, BF, [1 << 27, 16, 2, 128]),
                                           vc=_t(pm, 9, BF, [1 << 27, 16, 2, 128])), INVALID),
    ("bf16 cache with a scale", lambda pm: dict(ks=_t(pm, 11, F32, [])), INVALID),
    ("fp8 cache without scales", lambda pm: _fp8_caches(pm) | dict(ks=None), INVALID),
    ("scale of two", lambda pm: _fp8_caches(pm) | dict(vs=_t(pm, 12, F32, [2])), INVALID),
    ("no error word", lambda pm: dict(err=0), INVALID),
])
def test_append_refuses(pm, name, change, status):
    assert _append(pm, {**_append_args(pm), **change(pm)}) == status, name


def test_append_other_head_dim(pm):
    a = _append_args(pm)
    for key, n, heads in (("q", 0, 8), ("k", 1, 2), ("v", 2, 2), ("qo", 6, 8), ("ko", 7, 2)):
        a[key] = _t(pm, n, BF, [4, heads, 96])
    a["cs"] = _t(pm, 4, F32, [64, 96])
    a["kc"], a["vc"] = (_t(pm, n, BF, [10, 16, 2, 96]) for n in (8, 9))
    assert _append(pm, a) == UNSUPPORTED


def test_append_of_nothing_is_ok(pm):
    a = _append_args(pm)
    for key, n, heads in (("q", 0, 8), ("k", 1, 2), ("v", 2, 2), ("qo", 6, 8), ("ko", 7, 2)):
        a[key] = _t(pm, n, BF, [0, heads, 128], ptr=0)
    a["pos"], a["slots"] = _t(pm, 3, I32, [0], ptr=0), _t(pm, 5, I32, [0], ptr=0)
    assert _append(pm, a) == 0
    assert _append(pm, {**a, **_fp8_caches(pm)}) == 0


def _decode_args(pm):
    B, Hq, Hk, D = 3, 8, 2, 128
    return dict(q=_t(pm, 0, BF, [B, Hq, D]), kc=_t(pm, 1, BF, [10, 16, Hk, D]),
                vc=_t(pm, 2, BF, [10, 16, Hk, D]), o=_t(pm, 3, BF, [B, Hq, D]),
                ptr=_t(pm, 4, I32, [B + 1]), idx=_t(pm, 5, I32, [10]), last=_t(pm, 6, I32, [B]),
                sm=0.1, ks=None, vs=None, lse=_t(pm, 7, F32, [B, Hq]), ws=BASE + (8 << 28),
                n=1 << 30)


def _decode(pm, a):
    return pm._lib.mla_gqa_decode(_r(a["q"]), _r(a["kc"]), _r(a["vc"]), _r(a["o"]), _r(a["ptr"]),
                                  _r(a["idx"]), _r(a["last"]), a["sm"], _r(a["ks"]), _r(a["vs"]),
                                  _r(a["lse"]), ctypes.c_void_p(a["ws"]), a["n"], None)


@pytest.mark.parametrize("name,change,status", [
    ("q type", lambda pm: dict(q=_t(pm, 0, F8, [3, 8, 128])), INVALID),
    ("heads not grouped", lambda pm: dict(q=_t(pm, 0, BF, [3, 7, 128]), o=_t(pm, 3, BF, [3, 7, 128]),
                                          lse=_t(pm, 7, F32, [3, 7])), INVALID),
    ("q width", lambda pm: dict(q=_t(pm, 0, BF, [3, 8, 64]), o=_t(pm, 3, BF, [3, 8, 64])), INVALID),
    ("o type", lambda pm: dict(o=_t(pm, 3, F8, [3, 8, 128])), INVALID),
    ("o columns apart", lambda pm: dict(o=_t(pm, 3, BF, [3, 8, 128], [2048, 256, 2])), INVALID),
    ("indptr length", lambda pm: dict(ptr=_t(pm, 4, I32, [3])), INVALID),
    ("indices type", lambda pm: dict(idx=_t(pm, 5, F32, [10])), INVALID),
    ("indices missing", lambda pm: dict(idx=None), INVALID),
    ("no last page lengths", lambda pm: dict(last=None), INVALID),
    ("lse strides", lambda pm: dict(lse=_t(pm, 7, F32, [3, 8], [16, 1])), INVALID),
    ("scale is NaN", lambda pm: dict(sm=float("nan")), INVALID),
    ("bf16 cache with a scale", lambda pm: dict(vs=_t(pm, 9, F32, [])), INVALID),
    ("workspace missing", lambda pm: dict(ws=0), INVALID),
    ("workspace base", lambda pm: dict(ws=BASE + 128), INVALID),
    ("workspace small", lambda pm: dict(n=256), SMALL),
    ("page size", lambda pm: dict(kc=_t(pm, 1, BF, [10, 12, 2, 128]),
                                  vc=_t(pm, 2, BF, [10, 12, 2, 128])), UNSUPPORTED),
])
def test_decode_refuses(pm, name, change, status):
    assert _decode(pm, {**_decode_args(pm), **change(pm)}) == status, name


def test_decode_workspace_size(pm):
    f = pm.mla_get_gqa_decode_workspace_size
    # two spans of eight rows (values, maximum, sum) for each of 304 CTAs, counters, header
    assert f(1, 32, 8, 128, 152) == 256 + 1280 + 2 * 304 * 8 * 130 * 4
    assert f(1, 32, 8, 128, 152) == f(4096, 32, 8, 128, 152)
    assert f(1, 16, 1, 64, 152) == 256 + 1280 + 2 * 304 * 16 * 66 * 4
    assert f(1, 64, 1, 64, 152) == 256 + 1280 + 2 * 304 * 32 * 66 * 4
    for bad in ((1, 7, 2, 128), (1, 0, 1, 128), (-1, 8, 2, 128), (1, 8, 2, 80)):
        with pytest.raises(pm.MlaError):
            f(*bad, 152)


def test_error_word_is_checked(pm):
    import torch
    x = torch.zeros(1)
    with pytest.raises(ValueError):
        pm.mla_gqa_rope_and_cache(x, x, x, x, x, 0, x, x, x, x, torch.zeros(1))


def _prompt_args(pm):
    Hq, Hk, D = 8, 2, 128
    return dict(q=_t(pm, 0, BF, [7, Hq, D]), k=_t(pm, 1, BF, [9, Hk, D]), v=_t(pm, 2, BF, [9, Hk, D]),
                o=_t(pm, 3, BF, [7, Hq, D]), qo=_t(pm, 4, I32, [3]), kv=_t(pm, 5, I32, [3]), sm=0.1,
                lse=_t(pm, 6, F32, [7, Hq]), err=BASE + (7 << 28))


def _prompt(pm, a):
    return pm._lib.mla_prompt_attention(_r(a["q"]), _r(a["k"]), _r(a["v"]), _r(a["o"]), _r(a["qo"]),
                                        _r(a["kv"]), a["sm"], _r(a["lse"]), ctypes.c_void_p(a["err"]),
                                        ctypes.c_void_p(a.get("ws")), a.get("n", 0), None)


@pytest.mark.parametrize("name,change,status", [
    ("q type", lambda pm: dict(q=_t(pm, 0, F32, [7, 8, 128])), INVALID),
    ("q missing", lambda pm: dict(q=None), INVALID),
    ("q head stride 0", lambda pm: dict(q=_t(pm, 0, BF, [7, 8, 128], [1024, 0, 1])), INVALID),
    ("k head stride 0", lambda pm: dict(k=_t(pm, 1, BF, [9, 2, 128], [256, 0, 1])), INVALID),
    ("k base", lambda pm: dict(k=_t(pm, 1, BF, [9, 2, 128], ptr=BASE + 2)), INVALID),
    ("heads not grouped", lambda pm: dict(k=_t(pm, 1, BF, [9, 3, 128]), v=_t(pm, 2, BF, [9, 3, 128])), INVALID),
    ("k and v lengths", lambda pm: dict(v=_t(pm, 2, BF, [8, 2, 128])), INVALID),
    ("o width", lambda pm: dict(o=_t(pm, 3, BF, [7, 8, 64])), INVALID),
    ("o type", lambda pm: dict(o=_t(pm, 3, F32, [7, 8, 128])), INVALID),
    ("indptr lengths differ", lambda pm: dict(kv=_t(pm, 5, I32, [4])), INVALID),
    ("indptr empty", lambda pm: dict(qo=_t(pm, 4, I32, [0])), INVALID),
    ("scale zero", lambda pm: dict(sm=0.0), INVALID),
    ("scale negative", lambda pm: dict(sm=-1.0), INVALID),
    ("scale NaN", lambda pm: dict(sm=float("nan")), INVALID),
    ("scale infinite", lambda pm: dict(sm=float("inf")), INVALID),
    ("lse shape", lambda pm: dict(lse=_t(pm, 6, F32, [7, 2])), INVALID),
    ("no error word", lambda pm: dict(err=0), INVALID),
    ("workspace base", lambda pm: dict(ws=BASE + 4, n=1 << 30), INVALID),
    ("head widths", lambda pm: dict(v=_t(pm, 2, BF, [9, 2, 64]), o=_t(pm, 3, BF, [7, 8, 64])), UNSUPPORTED),
    ("group too large", lambda pm: dict(q=_t(pm, 0, BF, [7, 258, 128]), o=_t(pm, 3, BF, [7, 258, 128]),
                                        lse=None), UNSUPPORTED),
])
def test_prompt_refuses(pm, name, change, status):
    assert _prompt(pm, {**_prompt_args(pm), **change(pm)}) == status, name


def test_prompt_of_nothing_is_ok(pm):
    a = _prompt_args(pm)
    a.update(q=_t(pm, 0, BF, [0, 8, 128], ptr=0), o=_t(pm, 3, BF, [0, 8, 128], ptr=0), lse=None)
    assert _prompt(pm, a) == 0
    assert _prompt(pm, {**_prompt_args(pm), "qo": _t(pm, 4, I32, [1]), "kv": _t(pm, 5, I32, [1])}) == 0


def test_prompt_workspace_size(pm):
    f = pm.mla_get_prompt_workspace_size
    # two parts a SM (maximum, sum and output of 256 rows in fp32) and less than 128 bytes
    for dv in (64, 128):
        parts = 2 * 152 * 256 * (dv + 2) * 4
        assert parts < f(20000, dv, 152) < parts + 152 * 128
    assert f(1920, 128, 152) == 0              # too short to be cut anywhere
    for bad in ((-1, 128), (100, 96)):
        with pytest.raises(pm.MlaError):
            f(*bad, 152)


def test_packed_descriptors_are_the_structure(pm):
    """The bytes a call passes are mla_tensor_t's (on CPU tensors: their device index is -1)."""
    import torch
    base = torch.zeros(5, 6, 7, 8, dtype=torch.bfloat16)
    for t in (base, base[:, 1:3], base[0].transpose(0, 1), base[0, 0, ::2], torch.zeros(()),
              torch.zeros(0, 3, dtype=torch.int32)):
        assert pm._packed(t, -1) == bytes(pm._desc(t))
    assert pm._packed(None, 0) is None
    for bad, error in ((3, TypeError), (base, ValueError), ("x", TypeError)):
        with pytest.raises(error):
            pm._packed(bad, 0)
    with pytest.raises(TypeError):
        pm._packed(torch.zeros(2, dtype=torch.float64), -1)
    with pytest.raises(ValueError):
        pm._packed(torch.zeros(1, 1, 1, 1, 1), -1)

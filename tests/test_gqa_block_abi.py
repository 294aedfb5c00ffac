"""Host-side refusals of the block-scaled entry points (CPU only: nothing is enqueued)."""
import ctypes

import pytest
import torch

from tests.test_gqa_abi import BASE, BF, F8, F32, I32, INVALID, SMALL, UNSUPPORTED, _r, _t


@pytest.fixture(scope="module")
def pm():
    import paged_mla_latent_gb300 as m
    return m


def _caches(pm, hk=2, d=128, n=10, ps=32, nb=2):
    return dict(kc=_t(pm, 8, F8, [n, ps, hk, d]), vc=_t(pm, 9, F8, [n, ps, hk, d]),
                ks=_t(pm, 10, F32, [n, nb, hk]), vs=_t(pm, 11, F32, [n, nb, hk]))


def _lists(pm, B=3):
    return dict(qo=_t(pm, 12, I32, [B + 1]), kv=_t(pm, 13, I32, [B + 1]), idx=_t(pm, 14, I32, [7]),
                last=_t(pm, 15, I32, [B]))


# changes that every entry point with caches refuses alike
CACHES = [
    ("cache type", lambda pm: dict(kc=_t(pm, 8, BF, [10, 32, 2, 128]), vc=_t(pm, 9, BF, [10, 32, 2, 128])), INVALID),
    ("cache types differ", lambda pm: dict(vc=_t(pm, 9, BF, [10, 32, 2, 128])), INVALID),
    ("cache strides", lambda pm: dict(kc=_t(pm, 8, F8, [10, 32, 2, 128], [8192, 264, 128, 1]),
                                      vc=_t(pm, 9, F8, [10, 32, 2, 128], [8192, 264, 128, 1])), INVALID),
    ("page size", lambda pm: _caches(pm, ps=24, nb=2), UNSUPPORTED),
    ("no scale", lambda pm: dict(ks=None), INVALID),
    ("scale type", lambda pm: dict(vs=_t(pm, 11, BF, [10, 2, 2])), INVALID),
    ("scale rank", lambda pm: dict(ks=_t(pm, 10, F32, []), vs=_t(pm, 11, F32, [])), INVALID),
    ("scale pages", lambda pm: dict(ks=_t(pm, 10, F32, [9, 2, 2]), vs=_t(pm, 11, F32, [9, 2, 2])), INVALID),
    ("scale heads", lambda pm: dict(ks=_t(pm, 10, F32, [10, 2, 3]), vs=_t(pm, 11, F32, [10, 2, 3])), INVALID),
    ("scale shapes differ", lambda pm: dict(vs=_t(pm, 11, F32, [10, 4, 2])), INVALID),
    ("scale strides differ", lambda pm: dict(vs=_t(pm, 11, F32, [10, 2, 2], [8, 4, 1])), INVALID),
    ("scales overlap", lambda pm: dict(ks=_t(pm, 10, F32, [10, 2, 2], [4, 1, 1]),
                                       vs=_t(pm, 11, F32, [10, 2, 2], [4, 1, 1])), INVALID),
    ("more blocks than slots", lambda pm: _caches(pm, nb=64), INVALID),
    ("blocks no power of two", lambda pm: _caches(pm, ps=128, nb=3), UNSUPPORTED),
    ("blocks too long", lambda pm: _caches(pm, ps=1024, nb=4), UNSUPPORTED),
    ("list type", lambda pm: dict(kv=_t(pm, 13, F32, [4])), INVALID),
    ("list length", lambda pm: dict(kv=_t(pm, 13, I32, [5])), INVALID),
    ("indices rank", lambda pm: dict(idx=_t(pm, 14, I32, [7, 1])), INVALID),
    ("no last page", lambda pm: dict(last=None), INVALID),
    ("last page length", lambda pm: dict(last=_t(pm, 15, I32, [4])), INVALID),
]


def _append(pm, **change):
    T, hq, hk, d = 4, 8, 2, 128
    a = dict(q=_t(pm, 0, BF, [T, hq, d]), k=_t(pm, 1, BF, [T, hk, d]), v=_t(pm, 2, BF, [T, hk, d]),
             pos=_t(pm, 3, I32, [T]), cs=_t(pm, 4, F32, [64, 128]), neox=1, qout=_t(pm, 5, BF, [T, hq, d]),
             kout=_t(pm, 6, BF, [T, hk, d]), err=BASE, **_caches(pm), **_lists(pm))
    a.update(change)
    return pm._lib.mla_gqa_block_append(
        _r(a["q"]), _r(a["k"]), _r(a["v"]), _r(a["pos"]), _r(a["cs"]), a["neox"], _r(a["qo"]), _r(a["kv"]),
        _r(a["idx"]), _r(a["last"]), _r(a["qout"]), _r(a["kout"]), _r(a["kc"]), _r(a["vc"]), _r(a["ks"]),
        _r(a["vs"]), ctypes.c_void_p(a["err"]), None)


@pytest.mark.parametrize("name,change,status", CACHES + [
    ("q type", lambda pm: dict(q=_t(pm, 0, F32, [4, 8, 128])), INVALID),
    ("q base", lambda pm: dict(q=_t(pm, 0, BF, [4, 8, 128], ptr=BASE + 8)), INVALID),
    ("k stride", lambda pm: dict(k=_t(pm, 1, BF, [4, 2, 128], [258, 128, 1])), INVALID),
    ("v tokens", lambda pm: dict(v=_t(pm, 2, BF, [5, 2, 128])), INVALID),
    ("heads not grouped", lambda pm: dict(q=_t(pm, 0, BF, [4, 7, 128])), INVALID),
    ("positions", lambda pm: dict(pos=_t(pm, 3, I32, [3])), INVALID),
    ("table width", lambda pm: dict(cs=_t(pm, 4, F32, [64, 24])), INVALID),
    ("neox", lambda pm: dict(neox=2), INVALID),
    ("q_out shape", lambda pm: dict(qout=_t(pm, 5, BF, [4, 7, 128])), INVALID),
    ("q_out rows overlap", lambda pm: dict(qout=_t(pm, 5, BF, [4, 8, 128], [1024, 64, 1])), INVALID),
    ("k_out rows overlap", lambda pm: dict(kout=_t(pm, 6, BF, [4, 2, 128], [0, 128, 1])), INVALID),
    ("qo missing", lambda pm: dict(qo=None), INVALID),
    ("no error word", lambda pm: dict(err=0), INVALID),
    ("width", lambda pm: dict(q=_t(pm, 0, BF, [4, 8, 256]), k=_t(pm, 1, BF, [4, 2, 256]),
                              v=_t(pm, 2, BF, [4, 2, 256]), qout=_t(pm, 5, BF, [4, 8, 256]),
                              kout=_t(pm, 6, BF, [4, 2, 256]), **_caches(pm, d=256)), UNSUPPORTED),
])
def test_append_refuses(pm, name, change, status):
    assert _append(pm, **change(pm)) == status


def test_append_of_nothing(pm):
    empty = {n: _t(pm, 0, BF, [0, h, 128], ptr=0) for n, h in (("q", 8), ("k", 2), ("v", 2), ("qout", 8), ("kout", 2))}
    assert _append(pm, **empty, pos=_t(pm, 3, I32, [0], ptr=0)) == 0
    assert _append(pm, kout=None, **{n: t for n, t in empty.items() if n != "kout"}, pos=_t(pm, 3, I32, [0])) == 0


def _gather(pm, **change):
    hk, d = 2, 128
    a = dict(rows=_t(pm, 0, I32, [4]), kn=_t(pm, 1, BF, [4, hk, d]), vn=_t(pm, 2, BF, [4, hk, d]),
             kr=_t(pm, 3, BF, [50, hk, d]), vr=_t(pm, 4, BF, [50, hk, d]), err=BASE, **_caches(pm), **_lists(pm))
    a.update(change)
    return pm._lib.mla_gqa_block_gather(
        _r(a["kc"]), _r(a["vc"]), _r(a["ks"]), _r(a["vs"]), _r(a["kv"]), _r(a["idx"]), _r(a["last"]),
        _r(a["rows"]), _r(a["qo"]), _r(a["kn"]), _r(a["vn"]), _r(a["kr"]), _r(a["vr"]),
        ctypes.c_void_p(a["err"]), None)


@pytest.mark.parametrize("name,change,status", CACHES + [
    ("rows type", lambda pm: dict(rows=_t(pm, 0, F32, [4])), INVALID),
    ("rows missing", lambda pm: dict(rows=None), INVALID),
    ("new keys without their lists", lambda pm: dict(qo=None), INVALID),
    ("new keys without values", lambda pm: dict(vn=None), INVALID),
    ("new values' heads", lambda pm: dict(vn=_t(pm, 2, BF, [4, 3, 128])), INVALID),
    ("new tokens differ", lambda pm: dict(vn=_t(pm, 2, BF, [5, 2, 128])), INVALID),
    ("output type", lambda pm: dict(kr=_t(pm, 3, F32, [50, 2, 128])), INVALID),
    ("outputs differ", lambda pm: dict(vr=_t(pm, 4, BF, [51, 2, 128])), INVALID),
    ("output base", lambda pm: dict(vr=_t(pm, 4, BF, [50, 2, 128], ptr=BASE + 4)), INVALID),
    ("output rows overlap", lambda pm: dict(kr=_t(pm, 3, BF, [50, 2, 128], [128, 128, 1])), INVALID),
    ("no error word", lambda pm: dict(err=0), INVALID),
])
def test_gather_refuses(pm, name, change, status):
    assert _gather(pm, **change(pm)) == status


def test_gather_of_nothing(pm):
    assert _gather(pm, kr=_t(pm, 3, BF, [0, 2, 128], ptr=0), vr=_t(pm, 4, BF, [0, 2, 128], ptr=0)) == 0


def _decode(pm, **change):
    T, hq, d = 5, 8, 128
    a = dict(q=_t(pm, 0, BF, [T, hq, d]), o=_t(pm, 1, BF, [T, hq, d]), lse=_t(pm, 2, F32, [T, hq]), max_q=3, sm=0.1,
             ws=BASE + (30 << 28), ws_bytes=1 << 30, **_caches(pm), **_lists(pm))
    a.update(change)
    return pm._lib.mla_gqa_block_decode(
        _r(a["q"]), _r(a["kc"]), _r(a["vc"]), _r(a["ks"]), _r(a["vs"]), _r(a["o"]), _r(a["qo"]), _r(a["kv"]),
        _r(a["idx"]), _r(a["last"]), a["max_q"], a["sm"], _r(a["lse"]), ctypes.c_void_p(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("name,change,status", CACHES + [
    ("q type", lambda pm: dict(q=_t(pm, 0, F32, [5, 8, 128])), INVALID),
    ("heads not grouped", lambda pm: dict(q=_t(pm, 0, BF, [5, 7, 128]), o=_t(pm, 1, BF, [5, 7, 128])), INVALID),
    ("o shape", lambda pm: dict(o=_t(pm, 1, BF, [4, 8, 128])), INVALID),
    ("o type", lambda pm: dict(o=_t(pm, 1, F8, [5, 8, 128])), INVALID),
    ("o rows overlap", lambda pm: dict(o=_t(pm, 1, BF, [5, 8, 128], [64, 128, 1])), INVALID),
    ("lse shape", lambda pm: dict(lse=_t(pm, 2, F32, [5, 7])), INVALID),
    ("lse stride", lambda pm: dict(lse=_t(pm, 2, F32, [5, 8], [16, 1])), INVALID),
    ("no tokens a request", lambda pm: dict(max_q=0), INVALID),
    ("too many tokens a request", lambda pm: dict(max_q=65), INVALID),
    ("scale of softmax", lambda pm: dict(sm=float("nan")), INVALID),
    ("qo missing", lambda pm: dict(qo=None), INVALID),
    ("no workspace", lambda pm: dict(ws=0), INVALID),
    ("workspace base", lambda pm: dict(ws=BASE + 64), INVALID),
    ("workspace size", lambda pm: dict(ws_bytes=4096), SMALL),
    ("width", lambda pm: dict(q=_t(pm, 0, BF, [5, 8, 192]), o=_t(pm, 1, BF, [5, 8, 192]), **_caches(pm, d=192)),
     UNSUPPORTED),
])
def test_decode_refuses(pm, name, change, status):
    assert _decode(pm, **change(pm)) == status


def test_decode_workspace_sizes(pm):
    size = lambda *a: pm.mla_get_gqa_block_decode_workspace_size(*a, num_sms=152)
    assert size(8, 2, 128, 1) <= size(8, 2, 128, 4) == size(8, 2, 128, 64)
    assert size(64, 8, 128) == size(16, 2, 128)
    for bad, status in (((0, 1, 128), 1), ((8, 3, 128), 1), ((8, 2, 0), 1), ((8, 2, 96), 2), ((2048, 2, 128), 1),
                        ((8, 2, 128, 0), 1), ((8, 2, 128, 65), 1)):
        with pytest.raises(pm.MlaError) as e:
            size(*bad)
        assert e.value.status == status


def _table(pm, **change):
    B = 3
    a = dict(seq=_t(pm, 0, I32, [B]), new=_t(pm, 1, I32, [B]), table=_t(pm, 2, I32, [B, 9]), ps=16,
             free=_t(pm, 3, I32, [20]), count=_t(pm, 4, I32, [1]), out=_t(pm, 5, I32, []), qo=_t(pm, 6, I32, [B + 1]),
             key=_t(pm, 7, I32, [B + 1]), kv=_t(pm, 8, I32, [B + 1]), idx=_t(pm, 9, I32, [27]), last=_t(pm, 10, I32, [B]),
             pos=_t(pm, 11, I32, [8]), slots=_t(pm, 12, I32, [8]), err=BASE)
    a.update(change)
    return pm._lib.mla_build_page_table(
        _r(a["seq"]), _r(a["new"]), _r(a["table"]), a["ps"], _r(a["free"]), _r(a["count"]), _r(a["out"]), _r(a["qo"]),
        _r(a["key"]), _r(a["kv"]), _r(a["idx"]), _r(a["last"]), _r(a["pos"]), _r(a["slots"]),
        ctypes.c_void_p(a["err"]), None)


@pytest.mark.parametrize("name,change,status", [
    ("lengths missing", lambda pm: dict(seq=None), INVALID),
    ("lengths type", lambda pm: dict(seq=_t(pm, 0, F32, [3])), INVALID),
    ("lengths stride", lambda pm: dict(new=_t(pm, 1, I32, [3], [2])), INVALID),
    ("new lengths", lambda pm: dict(new=_t(pm, 1, I32, [4])), INVALID),
    ("table rank", lambda pm: dict(table=_t(pm, 2, I32, [27])), INVALID),
    ("table rows", lambda pm: dict(table=_t(pm, 2, I32, [4, 9])), INVALID),
    ("table columns apart", lambda pm: dict(table=_t(pm, 2, I32, [3, 9], [18, 2])), INVALID),
    ("table rows overlap", lambda pm: dict(table=_t(pm, 2, I32, [3, 9], [8, 1])), INVALID),
    ("page size", lambda pm: dict(ps=0), INVALID),
    ("page size no power of two", lambda pm: dict(ps=24), UNSUPPORTED),
    ("page too large", lambda pm: dict(ps=2048), UNSUPPORTED),
    ("positions past 31 bits", lambda pm: dict(table=_t(pm, 2, I32, [3, 1 << 21]), ps=1024), INVALID),
    ("pool without a count", lambda pm: dict(count=None), INVALID),
    ("pool without the new count", lambda pm: dict(out=None), INVALID),
    ("count without a pool", lambda pm: dict(free=None), INVALID),
    ("count of two", lambda pm: dict(count=_t(pm, 4, I32, [2])), INVALID),
    ("qo length", lambda pm: dict(qo=_t(pm, 6, I32, [3])), INVALID),
    ("keys missing", lambda pm: dict(key=None), INVALID),
    ("kv type", lambda pm: dict(kv=_t(pm, 8, F32, [4])), INVALID),
    ("indices rank", lambda pm: dict(idx=_t(pm, 9, I32, [27, 1])), INVALID),
    ("last length", lambda pm: dict(last=_t(pm, 10, I32, [2])), INVALID),
    ("positions without slots", lambda pm: dict(slots=None), INVALID),
    ("slots' length", lambda pm: dict(slots=_t(pm, 12, I32, [9])), INVALID),
    ("no error word", lambda pm: dict(err=0), INVALID),
    ("too many requests", lambda pm: dict(
        seq=_t(pm, 0, I32, [16385]), new=_t(pm, 1, I32, [16385]), table=_t(pm, 2, I32, [16385, 1]),
        qo=_t(pm, 6, I32, [16386]), key=_t(pm, 7, I32, [16386]), kv=_t(pm, 8, I32, [16386]),
        last=_t(pm, 10, I32, [16385])), UNSUPPORTED),
])
def test_table_refuses(pm, name, change, status):
    assert _table(pm, **change(pm)) == status


# ------------------------------------------------------------- the Python calls' own checks

def test_calls_refuse_cpu_tensors(pm):
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    n = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pm.mla_gqa_block_append(x, x, x, n, x, 1, n, n, n, n, x, x, x, x, x, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pm.mla_gqa_block_gather(x, x, x, x, n, n, n, n, x, x, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pm.mla_gqa_block_decode(x, x, x, x, x, x, n, n, n, n, 1, 1.0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pm.mla_build_page_table(n, n, n, 1, n, n, n, n, n, n)


@pytest.mark.parametrize("args,kind,text", [
    ((), TypeError, "arguments"),
    ((0,) + (None,) * 15, TypeError, "arguments"),
    ((0, "x") + (None,) * 15, TypeError, "torch.Tensor"),
    ((0, torch.zeros(3)) + (None,) * 15, ValueError, "CUDA device 0"),
])
def test_native_calls_check_their_arguments(pm, args, kind, text):
    with pytest.raises(kind, match=text):
        pm._native.mla_build_page_table(*args)


def test_native_calls_pass_statuses_on(pm):
    """None for every descriptor: the library's own refusal."""
    n = (None,) * 3
    with pytest.raises(ValueError, match="error_word"):
        pm._native.mla_build_page_table(0, *n, 16, *(None,) * 10, None, 0)
    assert pm._native.mla_gqa_block_decode(0, *(None,) * 10, 1, 1.0, None, 0, 0, 0) == INVALID
    with pytest.raises(OverflowError):
        pm._native.mla_gqa_block_decode(0, *(None,) * 10, 1 << 40, 1.0, None, 0, 0, 0)
    with pytest.raises(TypeError):
        pm._native.mla_gqa_block_decode(0, *(None,) * 10, 1, "x", None, 0, 0, 0)


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 1."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_tensors_device(pm, monkeypatch, current):
    """With either device current the library is called with the tensors' one (stand-ins: nothing
    is launched)."""
    now, calls = [current], []

    class Switch:
        def __init__(self, device):
            self.index = device if isinstance(device, int) else device.index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Native:
        def __getattr__(self, name):
            return lambda device, *args: calls.append((name, now[0], device)) or 0

    monkeypatch.setattr(pm, "_native", Native())
    monkeypatch.setattr(pm, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Switch)
    x = torch.Tensor._make_subclass(OnDevice, torch.zeros(4, 8, 128, dtype=torch.bfloat16))
    n = torch.Tensor._make_subclass(OnDevice, torch.zeros(4, dtype=torch.int32))
    pm.mla_build_page_table(n, n, n, 16, n, n, n, n, n, n, stream=7)
    pm.mla_gqa_block_append(x, x, x, n, x, 1, n, n, n, n, x, x, x, x, x, n, stream=7)
    pm.mla_gqa_block_gather(x, x, x, x, n, n, n, n, x, x, n, stream=7)
    pm.mla_gqa_block_decode(x, x, x, x, x, x, n, n, n, n, 1, 1.0, workspace=n, stream=7)
    assert [c[1:] for c in calls] == [(1, 1)] * 4 and now == [current]
    with pytest.raises(ValueError, match="workspace"):
        pm.mla_gqa_block_decode(x, x, x, x, x, x, n, n, n, n, 1, 1.0, workspace=torch.zeros(4), stream=7)

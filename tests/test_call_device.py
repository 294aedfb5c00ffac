"""Calls run on their tensors' device, whichever one is current (CPU only: the library and
torch's current device are stand-ins, nothing is launched)."""
import ctypes

import pytest
import torch


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 1."""
    index = 1

    @staticmethod
    def make(*shape, dtype=torch.bfloat16):
        return torch.Tensor._make_subclass(OnDevice, torch.zeros(*shape, dtype=dtype))

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


class Library:
    """Every function succeeds and notes the device that was current."""

    def __init__(self, current):
        self.current, self.calls = current, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current[0]))
            if "workspace_size" in name:
                ctypes.cast(args[-1], ctypes.POINTER(ctypes.c_size_t))[0] = 256
            return 0
        return call


@pytest.fixture(params=[0, 1])
def world(request, monkeypatch):
    """(module, library, [current device]) with device 0 or 1 current."""
    import paged_mla_latent_gb300 as pm
    current = [request.param]

    class Switch:
        def __init__(self, device):
            self.index = device if isinstance(device, int) else device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    lib = Library(current)
    monkeypatch.setattr(pm, "_lib", lib)
    monkeypatch.setattr(pm, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Switch)
    yield pm, lib, current
    assert current == [request.param]            # the caller's device is current again


def _i32(n):
    return OnDevice.make(n, dtype=torch.int32)


def _check(lib, *names):
    assert [n for n, _ in lib.calls] == list(names)
    assert all(device == 1 for _, device in lib.calls), lib.calls


def test_append(world):
    pm, lib, _ = world
    q, k = OnDevice.make(2, 4, 64), OnDevice.make(2, 2, 64)
    cache = OnDevice.make(3, 16, 2, 64)
    pm.mla_gqa_rope_and_cache(q, k, k, _i32(2), OnDevice.make(8, 64, dtype=torch.float32), 1, _i32(2), q,
                              cache, cache, _i32(1), k_out=k, stream=7)
    _check(lib, "mla_gqa_rope_and_cache")


def test_decode(world):
    pm, lib, _ = world
    q, cache = OnDevice.make(2, 4, 64), OnDevice.make(3, 16, 2, 64)
    ws = OnDevice.make(256, dtype=torch.uint8)
    pm.mla_gqa_decode(q, cache, cache, q, _i32(3), _i32(3), _i32(2), 0.1, workspace=ws, stream=7)
    _check(lib, "mla_gqa_decode")


def test_prompt(world):
    pm, lib, _ = world
    q, k = OnDevice.make(2, 4, 64), OnDevice.make(2, 2, 64)
    ws = OnDevice.make(256, dtype=torch.uint8)
    pm.mla_prompt_attention(q, k, k, q, _i32(2), _i32(2), 0.1, _i32(1), workspace=ws, stream=7)
    _check(lib, "mla_prompt_attention")


def test_prompt_makes_its_workspace_for_the_tensors_device(world, monkeypatch):
    """Its size depends on the device's SMs."""
    pm, lib, _ = world
    q, k = OnDevice.make(2, 4, 64), OnDevice.make(2, 2, 64)
    made = []
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: made.append((n, device)) or
                        OnDevice.make(n, dtype=dtype))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    pm.mla_prompt_attention(q, k, k, q, _i32(2), _i32(2), 0.1, _i32(1))
    _check(lib, "mla_get_prompt_workspace_size", "mla_prompt_attention")
    assert made == [(256, torch.device("cuda", 1))]


def test_latent_decode(world):
    """The latent entry points, the prepared call and the checks of a workspace."""
    pm, lib, _ = world
    q, kv = OnDevice.make(2, 4, 576), OnDevice.make(8, 576)
    ws, f = OnDevice.make(256, dtype=torch.uint8), OnDevice.make(1, dtype=torch.float32)
    args = (q, kv, q, _i32(3), _i32(3), _i32(8), _i32(2), 1, 0.1, f, f)
    pm.mla_decode(*args, workspace=ws, stream=7)
    pm.mla_decode_shared_prefix(*args, 2, workspace=ws, stream=7)
    pm.mla_decode_noalloc(*args, stream=7)
    pm.PreparedDecode(*args, workspace=ws, stream=7).run()
    pm.PreparedDecode(*args, workspace=ws, stream=7, compact_page_table=(_i32(1), _i32(3), _i32(2))).run()
    pm.mla_validate(*args[:2], *args[3:7], ws, stream=7)
    pm.mla_check_error(ws, stream=7)
    _check(lib, "mla_decode", "mla_decode_shared_prefix", "mla_decode_noalloc", "mla_decode",
           "mla_expand_shared_prefix_indices", "mla_decode", "mla_validate", "mla_check_error")


def test_latent_steps_around_the_decode(world):
    pm, lib, _ = world
    x, i = OnDevice.make(2, 4, 64), _i32(2)
    pm.mla_qk_rope_concat_and_cache(x, x, x, x, i, x, 0, i, x, x, x, x, _i32(1), stream=7)
    pm.mla_latent_to_v(x, x, x, stream=7)
    pm.mla_merge_partials(x, x, i, i, x, stream=7)
    pm.mla_expand_shared_prefix_indices(i, i, i, i, i, stream=7)
    pm.mla_selftest_bounded_wait(_i32(1), _i32(3), 1000, stream=7)
    _check(lib, "mla_qk_rope_concat_and_cache", "mla_latent_to_v", "mla_merge_partials",
           "mla_expand_shared_prefix_indices", "mla_selftest_bounded_wait")

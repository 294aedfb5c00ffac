"""The join of cut units on parts made by hand (tests/native/prompt_join_probe.cu): the sum in
the spans' order, and nothing where a CTA's wait ran out, whose part may be missing."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "native", "prompt_join_probe.cu")
LIB = os.path.join(HERE, "native", "_build", "libpromptjoinprobe.so")


@pytest.fixture(scope="module")
def probe():
    from paged_mla_latent_gb300 import build
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    tmp = LIB + f".{os.getpid()}"
    subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", tmp, SRC], check=True)
    os.replace(tmp, LIB)
    lib = ctypes.CDLL(LIB)
    lib.prompt_join_probe.restype = ctypes.c_int
    lib.prompt_join_probe.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]

    def run(spans, gave_up):
        o = np.full((256, 64), 0x7FC0, dtype=np.uint16)
        lse = np.full(256, np.nan, dtype=np.float32)
        n = lib.prompt_join_probe(spans, gave_up, o.ctypes.data, lse.ctypes.data)
        assert n > 1, n
        return n, (o.astype(np.uint32) << 16).view(np.float32), lse
    return run


@pytest.mark.parametrize("spans", [2, 5, 152, 300])
def test_join(probe, spans):
    n, o, lse = probe(spans, -1)
    # n parts of weight 1 and values 1 .. n: their mean, and ln n (fp32 sums of n terms, bf16)
    mean = (n + 1) / 2
    assert (np.abs(o - mean) <= mean * (2.0 ** -8 + n * 2.0 ** -24)).all()
    assert (np.abs(lse - np.log(n)) <= 2.0 ** -20 * np.log(n)).all()


@pytest.mark.parametrize("spans,gave_up", [(2, 0), (2, 1), (5, 2), (152, 0), (152, 77), (300, 299)])
def test_nothing_is_joined_after_a_wait_ran_out(probe, spans, gave_up):
    _, o, lse = probe(spans, gave_up)
    assert np.isnan(o).all() and np.isnan(lse).all()

"""The package where the compiled call module is missing (CPU only)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "paged_mla_latent_gb300"


@pytest.fixture
def without(tmp_path):
    """A copy of the package with its library, whose call module is not built and cannot be."""
    import paged_mla_latent_gb300 as pm
    shutil.copytree(os.path.join(ROOT, NAME), tmp_path / NAME,
                    ignore=shutil.ignore_patterns("_build", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    os.mkdir(tmp_path / NAME / "_build")
    (tmp_path / NAME / "csrc" / "native_calls.cpp").write_text("no C++")
    shutil.copy2(pm.library_path(), tmp_path / NAME / "_build")

    def run(code):
        r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                           env={k: v for k, v in os.environ.items() if k != "PYTHONPATH"})
        assert r.returncode == 0, r.stderr
        return r.stdout
    return run


def test_package_imports_without_the_call_module(without):
    """All but the calls that go through it work; those say what is missing."""
    out = without('''
import torch, paged_mla_latent_gb300 as pm
print(pm.mla_status_string(0), pm.mla_get_gqa_decode_workspace_size(1, 8, 1, 128, num_sms=152) > 0)
pm._cuda_index = lambda t: 0
pm._current_device = lambda: 0
pm._raw_stream = lambda stream, d: 0
n, e = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
for call in (lambda: pm.mla_build_page_table(n, n, n, 16, n, n, n, n, n, e),
             lambda: pm.mla_gqa_block_append(*[n] * 16), lambda: pm.mla_gqa_block_gather(*[n] * 11)):
    try:
        call()
    except ImportError as x:
        print("missing" if "pmla_native" in str(x) else x)
''')
    assert out.split() == ["MLA_OK", "True"] + ["missing"] * 3


def test_a_missing_call_module_rebuilds_nothing_else(without):
    out = without(f'''
import importlib.util
spec = importlib.util.spec_from_file_location("build", "{NAME}/build.py")
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
print(build.library_up_to_date(), build.native_up_to_date(), build.up_to_date())
''')
    assert out.split() == ["True", "False", "False"]


def test_a_call_module_that_does_not_build_leaves_the_library(without):
    """The library is in place before the module's failure is raised."""
    out = without(f'''
import importlib.util, os
spec = importlib.util.spec_from_file_location("build", "{NAME}/build.py")
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
one = os.path.join(build.CSRC, "mla_selftest.cu")
build._sources = lambda: [one]
os.remove(build.LIB_PATH)
try:
    build.build()
except RuntimeError as e:
    print("g++" in str(e), os.path.exists(build.LIB_PATH))
''')
    assert out.split() == ["True", "True"]

"""The C library builds, and counts as built, without the PyTorch extension."""
import importlib.util
import os
import pathlib
import shutil
import subprocess
import sys

import pytest

ROOT = pathlib.Path(__file__).resolve().parents[1]
PACKAGE = ROOT / "bit_kv_cache_nvfp4_gb300"

WITHOUT_TORCH = """
import importlib.util, sys
sys.modules["torch"] = None                      # any import of it raises
spec = importlib.util.spec_from_file_location("kv4_build", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
print(b.build())
"""


@pytest.fixture
def tiny(tmp_path):
    """A copy of the build file with a library of one small source."""
    package = tmp_path / "bit_kv_cache_nvfp4_gb300"
    (package / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "kv4mla.h").write_text("int kv4_answer(void);\n")
    shutil.copy(PACKAGE / "build.py", package / "build.py")
    text = (package / "build.py").read_text()
    start, end = text.index("SOURCES = ["), text.index("ARCH = [")
    (package / "build.py").write_text(text[:start] + 'SOURCES = ["one.cu"]\nHEADERS = []\n' + text[end:])
    (package / "csrc" / "one.cu").write_text('extern "C" int kv4_answer(void) { return 42; }\n')
    (package / "csrc" / "kv4_torch.cpp").write_text("this does not compile\n")
    spec = importlib.util.spec_from_file_location("kv4_tiny_build", package / "build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def need_nvcc():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("needs nvcc")


def test_library_is_built_without_pytorch(tiny):
    need_nvcc()
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH, tiny.__file__], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[-1] == tiny.LIB_PATH and os.path.exists(tiny.LIB_PATH)
    assert not os.path.exists(tiny.TORCH_PATH)


def test_a_broken_extension_leaves_the_library(tiny, capfd):
    need_nvcc()
    with pytest.raises(RuntimeError, match="kv4_torch.cpp"):
        tiny.build()
    capfd.readouterr()
    assert os.path.exists(tiny.LIB_PATH) and not tiny._stale()
    assert not os.path.exists(tiny.TORCH_PATH)
    made = os.path.getmtime(tiny.LIB_PATH)
    assert tiny.build_library() == tiny.LIB_PATH and os.path.getmtime(tiny.LIB_PATH) == made


def test_a_newer_extension_source_does_not_rebuild_the_library(tiny):
    need_nvcc()
    tiny.build_library()
    later = os.path.getmtime(tiny.LIB_PATH) + 10
    os.utime(os.path.join(tiny.CSRC, tiny.TORCH_SOURCE), (later, later))
    assert not tiny._stale() and tiny._torch_stale()

"""The package without its second binary, the binding of the row-wise operators."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "moe_grouped_gemm_03_b200")

CALLS = """
import torch
import moe_grouped_gemm_03_b200 as dg

assert dg.get_m_total_bound(3, 8) == 384 and dg.get_tma_aligned_size(5, 4) == 8
x = torch.zeros(4, 256)
for call in (lambda: dg.fp8_gemm_nt((x, x), (x, x), x),):  # refused for its types, not for a missing binary
    try:
        call()
    except ImportError:
        raise SystemExit("a GEMM needs the binding")
    except (dg.DGError, ValueError, TypeError):
        pass
for call in (lambda: dg.moe_permute(x, x, x), lambda: dg.rms_norm(x, x, x), lambda: dg.swiglu(x, x)):
    try:
        call()
    except ImportError as e:
        assert "_rowwise.so" in str(e) and "build" in str(e), e
    else:
        raise SystemExit("a row-wise operator ran without its binding")
"""


@pytest.mark.parametrize("binding", ["missing", "unreadable"])
def test_the_gemms_need_no_binding(tmp_path, binding):
    """libdg.so alone serves the GEMMs; the other operators say what is missing when they are called."""
    at = tmp_path / "moe_grouped_gemm_03_b200"
    at.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith((".py", "libdg.so")):
            shutil.copy(os.path.join(PACKAGE, name), at)
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    if binding == "unreadable":
        (at / "_rowwise.so").write_bytes(b"not a library")
    done = subprocess.run([sys.executable, "-c", CALLS], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_the_library_builds_without_torch(tmp_path):
    """Where torch is not installed the library is built (here: found up to date) and the binding left out."""
    code = f"""
import importlib.util, os, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("dg_build", {os.path.join(PACKAGE, "build.py")!r})
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
build.BINDING = {str(tmp_path / "_rowwise.so")!r}
assert build.build() == build.LIB and not os.path.exists(build.BINDING)
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
    assert "is not built" in done.stderr

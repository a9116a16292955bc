"""The gradient norm, clipping, all-reduce with norm and AdamW calls from
plain C (tests/c/grads_from_c.c): the header compiles as C99 and every check
comes before any device work."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "gradient_all_reduce_allreduce_amd")


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_c_program_calls_the_gradient_operators(tmp_path):
    if not os.path.exists(os.path.join(PKG, "libddp_allreduce.so")):
        pytest.fail("libddp_allreduce.so is not built")
    exe = str(tmp_path / "grads_from_c")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "grads_from_c.c"), "-o", exe, "-L", PKG,
                    "-lddp_allreduce", "-lm", "-Wl,-rpath," + PKG], check=True, capture_output=True, text=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, HIP_VISIBLE_DEVICES=""))
    assert p.returncode == 0, p.stdout + p.stderr
    assert "all checks passed" in p.stdout

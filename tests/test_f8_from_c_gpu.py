"""The 8-bit entry points from a plain C program (tests/f8_from_c.c),
built with the host C compiler against include/attn_res.h."""
import os
import subprocess

import pytest

from attention_residual_fusion_gb300 import _build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_f8_from_plain_c(tmp_path):
    lib = _build.build()
    exe = str(tmp_path / "f8_from_c")
    cmd = ["gcc", "-std=c11", "-O2", "-Wall", "-Werror", "-o", exe, os.path.join(ROOT, "tests", "f8_from_c.c"),
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(CUDA, "include")]
    for d in (os.path.dirname(lib), os.path.join(CUDA, "lib64")):
        cmd += ["-L", d, f"-Wl,-rpath,{d}"]
    r = subprocess.run(cmd + ["-lattn_res", "-lcudart", "-lm"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr

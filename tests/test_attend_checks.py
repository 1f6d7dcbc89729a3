"""Host-side checks of the attention kernel's bookkeeping: a small program
(``tests/attend_checks.cu``) around the functions that the kernels themselves
call, compiled by nvcc and run on the host."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_attend_checks(tmp_path):
    from deepseek_sparse_attention_row_gb300 import _build_lib

    exe = str(tmp_path / "attend_checks")
    cmd = [_build_lib.nvcc(), *_build_lib.ARCH, "-std=c++17", "-O2", "-I", _build_lib.CSRC,
           os.path.join(ROOT, "tests", "attend_checks.cu"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout + res.stderr

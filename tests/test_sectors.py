"""Rows on 32-byte boundaries (cp_geometry.h): plain C++, on the CPU; and that the projection asks for
them by that rule, which leaves arrays out that are not there."""
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
CSRC = ROOT / "trellis_row_decode_gb300" / "csrc"


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_rows_that_are_not_there_do_not_count(tmp_path):
    exe = tmp_path / "sectors"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", "-o", str(exe),
                    str(ROOT / "tests" / "sanitize" / "sectors_main.cpp")], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr
    assert "sectors ok" in run.stdout


def test_the_projection_asks_for_rows_by_that_rule():
    text = (CSRC / "cp_linear.cu").read_text()
    for array in ("out, out_stride", "residual, residual_stride", "pre, pre_stride"):
        assert f"sectors_ok({array}" in text

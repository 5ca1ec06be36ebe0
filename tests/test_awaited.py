"""What a warp that ends early waits for on its own barrier (cp_ring.h): plain C++, on the CPU; and that
the product's kernel keeps to it."""
import re
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
CSRC = ROOT / "trellis_row_decode_gb300" / "csrc"


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_a_load_whose_wait_ran_out_is_waited_for(tmp_path):
    exe = tmp_path / "awaited"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", "-o", str(exe),
                    str(ROOT / "tests" / "sanitize" / "awaited_main.cpp")], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr
    assert "awaited ok" in run.stdout


def test_residuals_are_waited_for_by_that_rule():
    """Each wait on the residual's barrier takes the parity from there, and one that ran out keeps the
    warp from the slot."""
    text = (CSRC / "cp_linear_tc.cu").read_text()
    waits = re.findall(r"mbar_wait\(residual_bar, ([^,]+),", text)
    assert waits == ["coming.parity"] * 2
    assert re.search(r"coming\.waited\(ok\);\s*if \(!ok\) return;", text)

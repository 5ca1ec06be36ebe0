"""What an 8-bit product waits for when it ends early (cp_ring.h): plain C++, on the CPU."""
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
CSRC = ROOT / "trellis_row_decode_gb300" / "csrc"


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_load_begun_is_waited_for(tmp_path):
    exe = tmp_path / "ring"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", "-o", str(exe),
                    str(ROOT / "tests" / "sanitize" / "ring_main.cpp")], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr
    assert "ring ok" in run.stdout

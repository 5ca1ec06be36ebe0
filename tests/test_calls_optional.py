"""The calls' compiled form is optional: without this Python's headers the library builds all the same, and
where the compiled code is missing or another machine's every call takes the checked way."""
import subprocess
import sys
import sysconfig
from pathlib import Path

import pytest
import torch

import trellis_row_decode_gb300 as cp
from trellis_row_decode_gb300 import build_ext, projection

ROOT = Path(__file__).resolve().parent.parent


@pytest.fixture(scope="module", autouse=True)
def built():
    if not (cp.LIB_PATH.exists() and build_ext.CALLS.exists()):
        build_ext.build()


def test_building_without_headers_leaves_no_calls(tmp_path, monkeypatch):
    calls = tmp_path / build_ext.CALLS.name
    calls.write_bytes(b"of another library")
    monkeypatch.setattr(build_ext, "CALLS", calls)
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert build_ext.build_calls() is None
    assert not calls.exists()


def test_building_with_headers_makes_them(tmp_path, monkeypatch):
    calls = tmp_path / build_ext.CALLS.name
    monkeypatch.setattr(build_ext, "CALLS", calls)
    assert build_ext.build_calls() == calls and calls.exists()
    assert [p.name for p in tmp_path.iterdir()] == [calls.name]


def test_the_calls_are_named_for_their_python():
    assert build_ext.CALLS.name == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert projection._CALLS_PATH == build_ext.CALLS


def test_the_package_leaves_its_build_alone():
    """`python -m trellis_row_decode_gb300.build_ext` runs a module that the package has not loaded."""
    code = "import sys, trellis_row_decode_gb300 as cp; print(cp.__name__ + '.build_ext' in sys.modules)"
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert run.stdout.strip() == "False", run.stderr


@pytest.mark.parametrize("content", [None, b"", b"\x7fELF of another machine"])
def test_missing_or_foreign_calls_are_done_without(tmp_path, monkeypatch, content):
    path = tmp_path / "_calls.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(projection, "_CALLS_PATH", path)
    monkeypatch.setattr(projection, "_calls", None)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        calls = projection._common()
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    assert calls.dropout(x, None, 0.1, 1, 2, None) is NotImplemented
    assert calls.linear(x, x) is NotImplemented and calls.linear_grad(x) is NotImplemented
    assert projection._common() is calls
    with pytest.raises(ValueError, match="CUDA"):              # the checked way, and its checks
        cp.linear(x, x)


@pytest.mark.gpu
def test_calls_without_the_compiled_form_are_the_same(monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda").bfloat16()
                for s in ((200, 72), (40, 72), (200, 40)))

    def run():
        out, pre = cp.linear(x, w, None, "gelu", p=0.2, seed=3, pre=True)
        return [out, pre, *cp.linear_grad(dy, x, w, "gelu", pre, p=0.2, seed=3),
                cp.dropout(x, 0.4, 5, residual=x)]
    assert projection._common() is not projection._Checked
    want = run()
    monkeypatch.setattr(projection, "_calls", projection._Checked)
    assert all(torch.equal(a, b) for a, b in zip(run(), want))

"""Every function of the instructions' header is called: nothing stays that no call reaches."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "trellis_row_decode_gb300" / "csrc"


def test_every_instruction_has_a_caller():
    text = (CSRC / "cp_tcgen05.cuh").read_text()
    names = re.findall(r"^__(?:device|host)__.*?(\w+)\(", text, re.M)
    assert len(names) > 30
    sources = "".join(p.read_text() for p in sorted(CSRC.glob("*.cu*")))
    for name in names:
        assert len(re.findall(rf"\b{name}\b(?:<[^>]*>)?\(", sources)) > 1, name

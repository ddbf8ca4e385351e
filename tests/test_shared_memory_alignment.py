"""Dynamic shared memory that is read or written 16 bytes at a time is declared so: what static shared memory lies before it is
the compiler's business, and an array of floats may begin on any 4 bytes."""
from __future__ import annotations

import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parent.parent / "combine_router_softmax_gb300" / "csrc"
BY_WORDS = {"route.cu", "layout.cu", "backward.cu"}  # whose shared memory is read value by value


def test_dynamic_shared_memory_is_aligned():
    seen = 0
    for path in sorted([*CSRC.glob("*.cu"), *CSRC.glob("*.cuh")]):
        text = path.read_text()
        for found in re.finditer(r"extern __shared__ (__align__\((\d+)\) )?([\w ]+?) ?(\w+)\[\];", text):
            seen += 1
            align, kind, name = int(found[2] or 0), found[3], found[4]
            rounded_up = f"smem_u32({name}) & 1023" in text
            assert align >= 16 or kind == "uint4" or rounded_up or path.name in BY_WORDS, f"{path.name}: {found[0]}"
    assert seen >= 16

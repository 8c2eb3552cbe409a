"""Dynamic shared memory starts behind a kernel's static arrays, at a multiple of what its declaration asks for.  Every array
that is read in 16-byte pieces asks for that itself, so that another static array before it cannot move it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_packed_varlen_causal_gb300", "csrc")


def declarations():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = open(path, encoding="utf-8").read()
        for kind, name in re.findall(r"extern __shared__ ([^;]*?)\b(\w+)\[\];", text):
            yield os.path.basename(path), kind.strip(), name, text


@pytest.mark.parametrize("file,kind,name", [d[:3] for d in declarations()])
def test_dynamic_shared_memory_asks_for_its_alignment(file, kind, name):
    text = next(d[3] for d in declarations() if d[:3] == (file, kind, name))
    align = re.search(r"__align__\((\d+)\)", kind)
    rounded = re.search(r"reinterpret_cast<uintptr_t>\(%s\)|smem_u32\(%s\)" % (name, name), text)      # placed by hand
    assert (align and int(align[1]) >= 16) or kind in ("uint4", "float4") or rounded


def test_there_are_some():
    assert len(list(declarations())) >= 5

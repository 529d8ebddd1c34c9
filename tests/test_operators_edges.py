"""What tests/test_operators.py leaves of include/emu_operators.h: the
alignment that the kernels' memory accesses claim, refusals of what autograd
would lose, and the paths that only large or unusual calls take."""
import os
import re
import subprocess

import pytest

from bit_exact_fp8_amd import build

ELEMENT = {"float": 4, "half": 2, "bfloat": 2}


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("source", ["emu_norm.hip", "emu_logprobs.hip"])
def test_rows_are_accessed_with_their_elements_alignment(source, tmp_path):
    """Rows begin at any element, so a vector of 8 of a row's elements is read
    and written with the element's alignment: what the compiler is told, in
    its own intermediate form of the kernels."""
    out = tmp_path / "kernels.ll"
    subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", "-emit-llvm", os.path.join(build.CSRC, source),
                    "-o", str(out)], check=True, capture_output=True)
    seen, wrong = {"load": 0, "store": 0}, []
    for line in out.read_text().splitlines():
        if not (m := re.search(r"\b(load|store) <8 x (float|half|bfloat)>.* addrspace\(1\).*, align (\d+)", line)):
            continue
        seen[m[1]] += 1
        if int(m[3]) > ELEMENT[m[2]]:
            wrong.append(line.strip())
    assert min(seen.values()) > 0
    assert not wrong, (len(wrong), wrong[:3])

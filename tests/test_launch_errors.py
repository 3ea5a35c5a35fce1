"""A call reports the error of its own launch, not one that a refused call before it
has left behind: no launch is judged by the runtime's last error."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "moe_decode_gemm_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h"))))
def test_no_launch_is_judged_by_the_last_error(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "<<<" not in text
    assert not re.search(r"(return|=|\()\s*cudaGetLastError\(", text)

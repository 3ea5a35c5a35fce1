"""A projection with 4-bit weights whose wait runs out gives no ring slot back that
it has not read: the slot's next copy would be issued while the last one is on its
way, the barrier's phases would no longer count copies, and a CTA could end, or
take its rings for the sums, before its copies have landed. No healthy run shows
it, so it is read off the kernel's source; what a stalled kernel does is run
in the index-checking build (test_w4_giveup_gpu)."""
import os
import re

import moe_decode_gemm_gb300 as dg
from conftest import ROOT

SOURCE = os.path.join(ROOT, "moe_decode_gemm_gb300", "csrc", "k_w4.cu")


def _mma_warp():
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("} else if (warp == 1) {")
    return text[start:text.index("} else {\n    \n    griddep_wait();", start)]


def test_no_slot_is_given_back_after_a_wait_that_ran_out():
    code = _mma_warp()
    loop = code[code.index("for (int kx"):code.index("s_flags[0] = 1")]
    waits = [m.start() for m in re.finditer(r"ok = mbar_wait\(", loop)]
    commits = [m.start() for m in re.finditer(r"umma_commit_elect\(", loop)]
    breaks = [m.start() for m in re.finditer(r"if \(!ok\) break;", loop)]
    assert len(waits) == 2 and len(commits) == 2
    # each wait is followed by a way out before anything else, and the outer loop's
    # commit by one after the inner loop
    for w in waits:
        end = loop.index(";", w) + 1
        assert re.match(r"\s*if \(!ok\) break;", loop[end:])
    assert any(commits[0] < b < commits[1] for b in breaks)


def test_stall_is_of_the_index_checking_build():
    from moe_decode_gemm_gb300 import build
    build.build()
    assert dg.lib().dec_debug_stall(1) == dg.DEC_EUNSUPPORTED
    dbg = dg._load(dg.DEBUG_LIB_PATH)
    assert dbg.dec_debug_stall(1) == 0
    assert dbg.dec_debug_stall(0) == 1 and dbg.dec_debug_stall(0) == 0

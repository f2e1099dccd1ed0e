"""Where a GEMM warp that gave up a bounded wait leaves its tile loop, read in the source.

A wait gives up by each lane's own clock, so at the limit some lanes of a warp may still see
the barrier complete.  What follows (shuffles with a full mask, tcgen05 loads, __syncwarp)
takes every lane: the epilogue may leave only by a decision that the warp shares.
"""
import os
import re

import nvfp4_precision_quantization_gb300 as nv

CSRC = os.path.join(os.path.dirname(nv.__file__), "csrc")


def _after(name, start, end):
    s = open(os.path.join(CSRC, name)).read()
    s = re.sub(r"//[^\n]*", "", s)
    i = s.index(start)
    return s[i:s.index(end, i)]


def _exits(code):
    """The conditions of the `break`s and `return`s in the code."""
    return [m.group(1) for m in re.finditer(r"if \(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)\s*"
                                            r"(?:break|return);", code)]


def test_tiled_epilogue_leaves_by_a_vote():
    # from the wait for the accumulator to the first thing that takes the whole warp
    code = _after("kernels_gemm.cu", "mbar_wait_bounded(acc_full, t & 1)", "if constexpr (EPI)")
    exits = _exits(code)
    assert len(exits) == code.count("break;") == 1
    assert exits[0].startswith("__any_sync(0xffffffffu,")


def test_few_rows_epilogue_leaves_by_a_vote():
    code = _after("kernels_gemm_few.cu", "const bool ready = mbar_wait_bounded(&acc_full[b]",
                  "tmem_ld16(")
    exits = _exits(code)
    assert len(exits) == code.count("break;") == 1
    assert exits[0].startswith("barrier_or<")

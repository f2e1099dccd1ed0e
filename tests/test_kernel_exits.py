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


def test_amax_and_encode_warps_leave_by_a_vote():
    # consumers of the amax pass, up to the first shuffle or __syncwarp
    code = _after("kernels_amax.cu", "mbar_wait_bounded(&full[s], (uint32_t)((k / kStages) & 1))",
                  "const uint8_t* stage = smem")
    assert _exits(code) == ["__any_sync(0xffffffffu, !ok || abort_flag)"]
    assert code.count("break;") == 1
    s = open(os.path.join(CSRC, "kernels_amax.cu")).read()
    assert "if (!__all_sync(0xffffffffu, mbar_wait_bounded(&col_bar[b], parity))) return false;" in s
    # the encode's producer warp and its consumers; with 16x16 blocks all consumers decide
    code = _after("kernels_quantize.cu", "mbar_wait_bounded(&empty[s],", "issue(k);")
    assert _exits(code) == ["__any_sync(0xffffffffu, !ok || abort_flag)"]
    code = _after("kernels_quantize.cu", "mbar_wait_bounded(&full[s], (uint32_t)((k / NS) & 1))",
                  "const uint8_t* stage = smem")
    assert _exits(code) == ["B2D ? consumer_any(!ok || abort_flag) : "
                            "__any_sync(0xffffffffu, !ok || abort_flag)"]
    assert code.count("break;") == 1 and "consumer_sync" not in code

"""Where a warp of the gated product that gave up a bounded wait leaves its loop, read in the
source: a wait gives up by each lane's own clock, and what follows (shuffles, tensor-memory
loads and stores, __syncwarp) takes every lane, so a warp leaves by a decision that it shares."""
from test_kernel_exits import _after, _exits


def test_epilogue_leaves_by_a_vote():
    # from the wait for the accumulators to the first shuffle or transposition
    code = _after("kernels_gated.cu", "mbar_wait_bounded(acc_full, t & 1)", "gated_block32<ALIGNED>(p")
    exits = _exits(code)
    assert code.count("break;") == 1
    # beside it, the loading lambda's end: which columns were loaded, the same for every lane
    assert exits == ["from + kHeld < kWarpCols", "__any_sync(0xffffffffu, !ready || *(volatile int*)err)"]


def test_scale_warps_leave_by_a_vote():
    code = _after("kernels_gated.cu", "bool ok = mbar_wait_bounded(&sf_full[s], ph)", "tmem_st16(")
    assert _exits(code) == ["__any_sync(0xffffffffu, !ok || *(volatile int*)err)"]
    assert code.count("break;") == 1


def test_the_pair_meets_before_it_leaves():
    """Nothing returns between the first and the last meeting of a pair's CTAs."""
    code = _after("kernels_gated.cu", "cluster_sync();", "pair_tmem_dealloc(tmem")
    assert "return;" not in code.replace("if (from + kHeld < kWarpCols) return;", "")
    assert code.count("cluster_sync();") == 2

"""CPU: what the memory model asks of the 4-bit kernels and no run can show, read from their sources."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_smoothquant_gemm_b200", "csrc")


def source(name):
    """A file's code, without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_arrivals_on_other_blocks_barriers_release():
    """An arrival at another block's barrier hands over memory that was read or written before it: only a release
    orders that, a dependency between the values does not."""
    names = [os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))]
    arrivals = [(n, m) for n in names for m in re.findall(r"mbarrier\.arrive\S*shared::cluster\S*", source(n))]
    assert any(n == "sq_tc.cuh" for n, _ in arrivals)
    assert [a for a in arrivals if ".release.cluster." not in a[1]] == []
    assert not [n for n in names if "relaxed" in source(n)]


def test_a_block_stays_for_sums_under_way_after_the_last_cluster_barrier():
    """When a wait has run out, sums that other blocks sent may still be coming.  The cluster barrier before the end says
    that all are sent, not that they are there: the time that they are given has to follow it."""
    text = source("sq_w4_tc.cu")
    kernel = text[text.index("w4_tc_kernel(const W4TcParams p)"):]
    kernel = kernel[:kernel.index("namespace sqh")]
    assert kernel.count("__nanosleep") == 1
    assert kernel.rindex("cluster_sync();") < kernel.index("__nanosleep")


def test_blocks_without_tiles_wait_for_their_copies():
    """A block of the gate/up kernel starts to copy the tokens before it knows whether it has a tile.  Without one it
    never comes to the wait inside the loop over its tiles, and must not leave with copies to its memory under way."""
    text = source("sq_moe.cu")
    kernel = text[text.index("moe_up_kernel(const MoeParams p)"):text.index("moe_down_kernel(const MoeParams p)")]
    assert kernel.index("moe_stage_rows(") < kernel.index("for (int p0 = 0;")
    assert kernel.rindex("p.h[") < kernel.rindex("cp_wait_all();")

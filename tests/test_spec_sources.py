"""Orderings that the tree-attention kernels have to state in their source: no run can be relied on to show them missing."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_kv_cache_quant_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_a_lanes_own_answer_on_a_barrier_never_branches_around_a_warps_wait():
    """role_wait_warp votes with all 32 lanes. A barrier may complete between two lanes' mbar_test, so a branch on such an
    answer has to be on the warp's vote of it, or some lanes stay in the vote for ever."""
    text = source("tree_tc_kernels.cu")
    own = set(re.findall(r"const bool (\w+) = [^;]*\bmbar_test\(", text))
    assert own
    guarded = [c for c in re.findall(r"\bif \(([^;{}]*)\) ok = role_wait_warp\(", text)]
    assert len(guarded) >= 3
    for condition in guarded:
        left = re.sub(r"__all_sync\(0xffffffffu, \w+\)", "", condition)
        assert not own & set(re.findall(r"\w+", left)), condition


def test_a_segment_that_one_lane_found_is_ordered_before_its_warps_reads():
    """One lane writes the warp's walk in shared memory and all lanes read it: a vote does not order memory."""
    body = re.search(r"auto next = \[&\]\(\) -> bool \{(.*?)\n  \};", source("tree_tc_kernels.cu"), re.S).group(1)
    written = body.index("next_here()")
    assert "__syncwarp()" in body[:written] and "__syncwarp()" in body[written:]


def test_the_second_pass_over_a_tile_stores_its_weights_after_the_firsts():
    """Stores to tensor memory are asynchronous: a second one to the same columns has to wait for the first, which in
    this path may hold infinities."""
    text = source("tree_tc_kernels.cu")
    again = re.search(r"if \(!fresh\) \{(.*?)#pragma unroll", text, re.S).group(1)
    assert "tmem_wait_st()" in again


def test_lanes_without_a_row_meet_their_warp_before_it_moves_tensor_memory():
    """tcgen05.ld and .st are the whole warp's: what only the lanes with a query row do stands between a __syncwarp and
    the one before."""
    text = source("tree_tc_kernels.cu")
    out = re.search(r"for \(int c0 = c_begin;.*?\{(.*?)tmem_ld16", text, re.S).group(1)
    assert "__syncwarp()" in out
    query = re.search(r"if \(live\) x = (.*?)tmem_st32", text, re.S).group(1)
    assert "__syncwarp()" in query


def test_what_the_headers_of_these_calls_define_is_used():
    files = {n: source(n) for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h"))}
    everything = "\n".join(files.values())
    for name in ("tc_device.cuh", "tree_plan.cuh", "spec_internal.h"):
        defined = re.findall(r"__forceinline__ [\w:<>]+ (\w+)\(", files[name]) + re.findall(r"constexpr \w+ (k[A-Z]\w*) =", files[name])
        assert defined
        for d in defined:
            assert len(re.findall(rf"\b{d}\b", everything)) > 1, f"{name}: {d}"


def test_limits_of_the_kernels_are_the_headers():
    """The kernels' shared arrays go by constants of their own, the host's checks by the public header's."""
    text = source("spec_api.cu")
    for own, public in (("kSpecMaxBatch", "KVQ_SPEC_MAX_BATCH"), ("kTreeMax", "KVQ_TREE_MAX")):
        assert re.search(rf"static_assert\([^;]*kvq::{own} == {public}\b", text), own


def test_the_allocating_warp_is_whole_when_it_allocates():
    """tcgen05.alloc is the whole warp's, and one lane has just written the warp's walk."""
    before = source("tree_tc_kernels.cu").split("tmem_alloc(", 1)[0]
    assert "__syncwarp()" in before[before.rindex("walk[warp].start(s)"):]

"""What orders the hand-offs of the tensor-core kernels, as their sources have it (no GPU)."""
import os
import re

import pytest

from test_block_scaled_host import CSRC, source

SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))


@pytest.mark.parametrize("name", SOURCES)
def test_another_ctas_barrier_is_told_at_cluster_scope(name):
    """A release at CTA scope (the default too) orders nothing for a thread of another CTA.  Relaxed arrivals hand back
    what has been read, and hand over no data."""
    for arrive in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster", source(name)):
        assert re.match(r"mbarrier\.arrive\.(release|relaxed)\.cluster\.shared::cluster", arrive), arrive


def test_converting_warps_arrive_within_their_cta():
    """The pair's converting warps and the leader's MMAs: a thread between them passes on what the other CTA has
    converted."""
    text = source("tc_linear_int8_many.cu")
    assert len(re.findall(r"mbar_arrive\(&converted\[unit\]\)", text)) == 2
    assert len(re.findall(r"mbar_arrive_remote_shared\(", text)) == 1 and "mbar_wait(&cpeer[unit], phase" in text
    assert re.search(r"void mbar_arrive_remote_shared.*?fence\.release\.sync_restrict::shared::cta\.cluster;.*?mbarrier\.arrive\.relaxed",
                     source("linear_int8_dev.cuh"), re.S)


@pytest.mark.parametrize("name,single", [("tc_linear_int8_few.cu", 1), ("tc_linear_int8_many.cu", 2)])
def test_warps_leave_their_waits_together(name, single):
    """Lanes that a wait lets go one by one are no warp for the TMEM accesses behind it.  `single`: the roles of one thread."""
    waits = [line for line in source(name).split("\n") if "goto teardown" in line]
    assert sum("whole_warp(" not in w and "next_tile(" not in w for w in waits) == single, waits
    for line in source(name).split("\n"):
        assert not re.search(r"\bif \(!\w+ && !mbar_wait", line), line


@pytest.mark.parametrize("name", ["tc_linear_int8_few.cu", "tc_linear_int8_many.cu"])
def test_a_stage_is_given_back_when_it_has_been_used(name):
    """Not when its bytes have been asked for: the copy that overwrites them starts at that arrival."""
    loops = [loop for loop in re.split(r"for \(int k = ", source(name)) if "mbar_arrive(&empty[stage])" in loop]
    assert len(loops) == 2
    for loop in loops:
        assert loop.index("mbar_arrive(&empty[stage])") > loop.rindex("f16_of_int8_16(")


@pytest.mark.parametrize("name", [f for f in SOURCES if "mbar_wait(&tfull" in source(f)])
def test_warps_that_read_accumulators_leave_their_wait_together(name):
    """Every kernel's epilogue: tcgen05.ld follows."""
    for wait in re.findall(r"[^\n]*mbar_wait\(&tfull[^\n]*\n[^\n]*", source(name)):
        assert "whole_warp(" in wait or wait.split("\n")[1].strip() == "__syncwarp();", wait


@pytest.mark.parametrize("name", ["linear_int8_dev.cuh", "tc_linear_int8_few.cu", "tc_linear_int8_many.cu"])
def test_accumulators_are_loaded_and_waited_for_in_one_statement(name):
    """In two, nothing keeps the compiler from using the registers between them."""
    assert not re.search(r"tmem_ld_32x32b_x\d+\(|tmem_ld_wait\(", source(name))

"""Waits that several warps of a kernel make together, in every order of their steps (CPU), and on
the device.

The warps that join parts of a tile (few_rows.cu) wait for a part, pass a barrier of all four
and go on; when their block has given up they leave for the barrier at the kernel's end.  The
model steps four warps, a producer that posts the part and a role that gives up, in every
order.  Where each warp goes by what it has seen itself, some orders end with warps at
different barriers, which never fill; where all meet and go by what all have seen, none does.
"""
from __future__ import annotations

import os
import re

import pytest

WARPS = 4


def stuck_orders(together: bool):
    """States that no step leads out of, short of all warps at the end."""
    # a warp waits ("poll"), is at the barrier of four with what it has seen ("join yes", "join no"),
    # at the barrier of the block ("end"), or has passed the one it was at ("done")
    start = (("poll",) * WARPS, False, False)          # warps, posted, given up
    seen, todo, stuck = {start}, [start], []
    while todo:
        warps, posted, aborted = state = todo.pop()
        steps = []
        if not posted:
            steps.append((warps, True, aborted))
        if not aborted:
            steps.append((warps, posted, True))
        for w, at in enumerate(warps):
            if at == "poll":
                moves = (["join yes"] if posted else []) + (["join no" if together else "end"] if aborted else [])
                steps += [(warps[:w] + (to,) + warps[w + 1:], posted, aborted) for to in moves]
        if all(at.startswith("join") for at in warps):
            steps.append((("done" if all(at == "join yes" for at in warps) else "end",) * WARPS, posted, aborted))
        if all(at == "end" for at in warps):
            steps.append((("done",) * WARPS, posted, aborted))
        if not steps and warps != ("done",) * WARPS:
            stuck.append(state)
        for s in steps:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return stuck


def test_warps_that_go_by_what_all_have_seen():
    assert not stuck_orders(together=True)


def test_the_model_sees_warps_that_go_by_what_each_has_seen():
    stuck = stuck_orders(together=False)
    assert stuck and all({"join yes", "end"} == set(warps) for warps, *_ in stuck)


@pytest.mark.gpu
@pytest.mark.parametrize("posted,aborted", [(True, False), (False, False), (False, True), (True, True)])
def test_threads_that_wait_together_go_on_or_stop_together(posted, aborted):
    from gshard_top_gating_b200 import _lib as L
    allowed = {L.MOE_OK} if posted and not aborted else {L.MOE_ERR_TIMEOUT} if not posted else {L.MOE_OK, L.MOE_ERR_TIMEOUT}
    for _ in range(20):
        assert L.moe_selftest_wait_together(posted, aborted, 2000) in allowed


def test_a_block_that_gave_up_lets_its_copies_land():
    """Each kernel with an abort flag goes through let_copies_land once, right before the barrier at
    its end and the release of its TMEM."""
    here = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gshard_top_gating_b200", "csrc")
    end = re.compile(r"let_copies_land\(abort_flag\);\n(?:  __syncwarp\(\);\n)?  (?:__syncthreads|cluster_sync_all)\(\);[^\n]*\n"
                     r"  if \(warp == 1\) \{\n    tc_fence_after\(\);\n    tmem_dealloc")
    kernels = 0
    for name in sorted(os.listdir(here)):
        if name.endswith(".cu"):
            with open(os.path.join(here, name)) as f:
                text = f.read()
            flags = text.count("volatile int* abort_flag = ")
            assert flags == len(end.findall(text)) == text.count("let_copies_land("), name
            kernels += flags
    assert kernels >= 10

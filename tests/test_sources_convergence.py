"""Source rules of the tensor-core kernels that no GPU is needed to check.

TMEM instructions are .sync.aligned: the whole warp has to execute them together.  A bounded wait
is a loop that every lane leaves by itself, so a warp that waits and goes on to such an instruction
(or to __syncwarp, which a lane that gave up elsewhere would never reach) does so through
mbar_wait_warp, and the Muon kernels converge directly before every group of TMEM instructions."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sample_gradient_clipping_b200", "csrc")
ENGINES = ("umma_gemm.cuh", "umma_gemm_2sm.cuh", "muon.cuh")


def _code(fn):
    """The file's lines without comments and blank ones."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, fn)).read())
    return [line.strip() for line in text.splitlines() if line.strip()]


@pytest.mark.parametrize("fn", ENGINES)
def test_whole_warps_wait_together(fn):
    """The accumulators' barriers (and the one-launch form's `done`) are waited for by whole warps."""
    waits = [line for line in _code(fn) if re.search(r"mbar_wait_\w+\(smem_addr\((acc_full|&done)", line)]
    assert waits and all("mbar_wait_warp(" in line for line in waits), waits


def test_tmem_instructions_of_converged_warps():
    code = _code("muon.cuh")
    sites = 0
    for k, line in enumerate(code):
        if not re.match(r"(tmem_ld32|tmem_st32|tmem_st_wait|tmem_alloc\w*)\(", line):
            continue
        sites += 1
        j = k - 1
        while re.match(r"(tmem_\w+\(|float .*;|const .*;)", code[j]):
            j -= 1
        if line.startswith("tmem_alloc") and code[j].startswith(("if constexpr (PAIR)", "} else {", "if (warp == 1)")):
            continue                              # a warp that has taken no branch of single lanes before
        assert "__syncwarp()" in code[j], (line, code[j])
    assert sites >= 12

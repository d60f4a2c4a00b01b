"""Hand-placed barriers of the HIP sources.  The barrier builtin alone orders
no memory access for the compiler, and neither does an asm wait in front of
it for what follows the barrier: an LDS access could be placed between the
two, before the other waves have arrived.  A wait and its barrier are
therefore one asm statement with a memory clobber, or the builtin is followed
at once by a scheduling fence."""
import glob
import os
import re

from sparse_expert_routing_sigmoid_amd import build as B


def code_lines(path):
    """The lines that are not only a comment, without their trailing comment."""
    with open(path) as f:
        lines = [re.sub(r"//.*", "", line).strip() for line in f]
    return [line for line in lines if line]


def test_barrier_builtins_are_fenced():
    bare = []
    for path in sorted(glob.glob(os.path.join(B.CSRC, "*"))):
        lines = code_lines(path)
        bare += [f"{os.path.basename(path)}: {lines[i - 1]} / {line}" for i, line in enumerate(lines)
                 if "__builtin_amdgcn_s_barrier()" in line
                 and "__builtin_amdgcn_sched_barrier(0)" not in lines[i + 1]]
    assert not bare, bare


def test_asm_barriers_wait_and_clobber():
    for path in sorted(glob.glob(os.path.join(B.CSRC, "*"))):
        for line in code_lines(path):
            if "asm" in line and "s_barrier" in line:
                assert "s_waitcnt" in line and '"memory"' in line, f"{os.path.basename(path)}: {line}"

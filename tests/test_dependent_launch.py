"""Kernels launched with programmatic stream serialisation start while the one
before them still runs, and see its writes, and those of what ran before it,
once they have executed griddepcontrol.wait themselves.  Read from the sources:
no such kernel signals, allocates tensor memory or touches global memory ahead
of grid_dep_wait()."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_xl_relative_txl_gb300",
                    "csrc")
KERNEL = re.compile(r"__global__ void __launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*(\w+)\(")
# What reads or writes global or tensor memory, or lets the next kernel start.
TOUCHES = re.compile(r"grid_dep_launch_dependents|tmem_alloc|tmem_ld|tmem_st|tma_load|tma_store|tma_reduce|plan_begin|"
                     r"run_tile_loader|atomic\w+\(|__ldg|cp_async|copy4|\bp\.(?:cuts|part|args\.(?:book|slots|cu|status))|"
                     r"\bb\.(?:table|start|rows|refs)\s*\[|read_slot|report_pages")


def kernels():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        if "launch_dependent(" not in text:
            continue
        for m in KERNEL.finditer(text):
            at = text.index("{", m.end())  # the body
            depth = 0
            for i in range(at, len(text)):
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                if depth == 0:
                    break
            out.append((os.path.basename(path), m.group(1), text[at:i]))
    return out


KERNELS = kernels()
PAGED = [k for k in KERNELS if k[0].startswith("page")]


def test_the_kernels_are_found():
    assert {k[1] for k in PAGED} >= {"paged_tc64_kernel", "paged_tc128_kernel", "paged_decode_kernel", "paged_simt_kernel",
                                     "paged_join_kernel", "reserve_kernel", "append_kernel", "copy_kernel", "fork_kernel",
                                     "free_kernel", "compact_kernel", "rename_kernel"}


@pytest.mark.parametrize("file,name,body", PAGED, ids=[k[1] for k in PAGED])
def test_nothing_is_touched_ahead_of_the_wait(file, name, body):
    ahead, wait, _ = body.partition("grid_dep_wait();")
    assert wait, "no wait"
    assert TOUCHES.findall(ahead) == []
    assert "return" not in ahead

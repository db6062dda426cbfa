"""Kernels launched while the one before them still runs wait for it before they read.

griddepcontrol.wait makes what earlier kernels wrote visible to the kernel that executes it, and to
no other: a kernel that reads memory before its own wait relies on somebody else's.  So in the source
of every kernel the wait is unconditional, stands before the trigger that lets the next kernel start,
and no memory is read above it.
"""

import glob
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "mixture_experts_layer_04_gb300", "csrc")
WAIT, TRIGGER = "grid_dep_wait();", "grid_dep_trigger();"
READS = re.compile(r"\.load\(|__ldg\(|\bload\w*\(|p\.offsets\[|\bcol\.vector\(")


def functions_with_a_trigger():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        lines = open(path, encoding="utf-8").read().split("\n")
        start = 0
        for i, line in enumerate(lines):
            if line.startswith("}"):
                body = lines[start:i]
                if any(TRIGGER in q for q in body):
                    yield f"{os.path.basename(path)}:{start + 1}", body
                start = i + 1


BODIES = list(functions_with_a_trigger())


def test_there_are_such_kernels():
    assert len(BODIES) > 25


@pytest.mark.parametrize("body", [b for _, b in BODIES], ids=[n for n, _ in BODIES])
def test_the_wait_comes_first(body):
    code = [q.split("//")[0].strip() for q in body]
    code = [q for q in code if q]
    waits = [i for i, q in enumerate(code) if WAIT in q]
    triggers = [i for i, q in enumerate(code) if TRIGGER in q]
    assert len(waits) == 1 and triggers
    assert code[waits[0]] == WAIT, "a conditional wait"
    assert triggers[0] > waits[0]
    opening = next(i for i, q in enumerate(code) if "__global__" in q or "__device__" in q)
    assert not [q for q in code[opening:waits[0]] if READS.search(q)]


@pytest.mark.parametrize("name", ["grouped_gemm.cu", "grouped.cu", "grouped_plan.cuh", "block_norm.cu",
                                  "grad_norm.cu"])
def test_no_read_only_loads_of_what_the_kernel_before_wrote(name):
    """ld.global.nc is for memory that nothing writes while the kernel runs, and these kernels run while
    the one before them still writes the plan (or a vector of a norm)."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        assert "__ldg" not in f.read()

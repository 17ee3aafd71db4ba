"""Programmatic dependent launch, read from the kernels' source: memory that an
earlier grid wrote is visible only to a grid that itself executes the dependency
wait, so every kernel does, in all of its threads and under no condition."""
import os
import re

from sparse_moe_layer_05_b200 import build as BUILD

SOURCES = [f for f in BUILD.SOURCES + BUILD.HEADERS if f != "moe_ptx.cuh"]


def lines_of(name):
    src = open(os.path.join(BUILD.CSRC, name)).read()
    return [line.split("//")[0].strip() for line in src.splitlines()]


def test_every_dependency_wait_is_unconditional():
    """A statement of its own, not behind an if on the same or the line before."""
    found = 0
    for name in SOURCES:
        lines = [x for x in lines_of(name) if x]
        for before, line in zip([""] + lines, lines):
            if "pdl_wait_and_trigger" in line:
                found += 1
                assert line == "pdl_wait_and_trigger();", (name, line)
                assert not re.match(r"(else\b|(\}\s*else\s+)?if\s*\(.*\)$)", before), (name, before)
    assert found >= 30


def test_every_kernel_of_the_training_calls_waits():
    for name in ("moe_router_grad.cu", "moe_router_grad_tc.cu", "moe_norm_ckpt.cu"):
        src = open(os.path.join(BUILD.CSRC, name)).read()
        assert len(re.findall(r"__global__", src)) == src.count("pdl_wait_and_trigger();"), name

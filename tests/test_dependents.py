"""Rules for kernels that may start beside whatever ran before them on the
stream: none reads memory before it has waited, and none through a path that
takes the data for constant while it runs.  (No run shows a breach for certain.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_03_gb300", "csrc")
# every launch in these is a dependent of the kernel before it, whichever that is
FILES = ["linear.cu", "gemv.cu", "adamw.cu"]


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(source):
    """name -> body of every __global__ function"""
    out = {}
    for m in re.finditer(r"__global__", source):
        name = re.search(r"(\w+_kernel)\s*\(", source[m.start():]).group(1)
        start = at = source.index("{", m.start())
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(source[at], 0)
            at += 1
            if depth == 0:
                break
        out[name] = source[start:at]
    return out


def test_the_kernels_are_found():
    assert len(kernels(text("linear.cu"))) >= 9 and "adamw_kernel" in kernels(text("adamw.cu"))


@pytest.mark.parametrize("name", FILES)
def test_every_kernel_waits_whatever_its_arguments(name):
    for kernel, body in kernels(text(name)).items():
        waits = [line for line in body.split("\n") if "pdl_wait()" in line]
        assert waits, kernel
        for line in waits:
            assert line.strip() == "pdl_wait();", f"{kernel}: {line.strip()}"


def test_no_launch_says_when_its_kernel_waits():
    # a parameter that says when is a kernel that may not wait first
    assert not re.search(r"\bwait_(end|start|at)\b", text("linear.cu"))


@pytest.mark.parametrize("name", FILES + ["fused.cuh", "pair_gemm.cuh", "launch.cuh"])
def test_no_load_takes_its_data_for_constant(name):
    # the kernel before may write it while this one runs already
    assert not re.search(r"ld\.global[\w.:]*\.nc\b|__ldg\s*\(|__restrict__", text(name))


def test_the_head_reads_what_an_earlier_kernel_of_the_call_left_from_l2():
    # head_target_kernel beside dh: g's kernel wrote lo, owner and hmax, dh's waited for it, this one only at its end
    body = kernels(text("head.cu"))["head_target_kernel"]
    for what in (r"\bowner\[", r"\blo\[", r"\bhmax\["):
        assert not re.search(what, body)
    assert body.count("__ldcg(") == 3

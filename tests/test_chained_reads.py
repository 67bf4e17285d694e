"""Kernels that are launched while the kernel before them still runs (those that call chain_wait) must
not read what that kernel writes through the non-coherent path: neither as a const __restrict__
parameter, which the compiler may turn into such loads, nor by __ldg.  Checked in the sources, since a
stale value shows only when the schedule happens to bring one."""

import os
import re

from fp16_gemm_relu_gb300 import build

# the caller's own inputs, and copies of them that are finished before the chain begins
INPUTS = {"index", "teacher", "dloss", "x", "w"}


def kernels():
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        for m in re.finditer(r"__global__.*?\n}\n", text, re.S):
            if "chain_wait()" in m.group(0):
                yield name, m.group(0)


def test_chained_kernels_read_coherently():
    seen = 0
    for name, text in kernels():
        seen += 1
        head, body = text.split("{", 1)
        for p in re.findall(r"const [\w ]+\* __restrict__ (\w+)", head):
            assert p in INPUTS, (name, head.split("(")[0].split()[-1], p)
        for arg in re.findall(r"__ldg\(([^;]*)", body):
            assert re.search(r"\bfrom\b", arg), (name, arg)  # x, as tg_head_grad_kernel calls it
    assert seen >= 7


def test_shared_epilogues_read_coherently():
    with open(os.path.join(build.CSRC, "tg_gemm_kernel.cuh")) as f:
        text = f.read()
    assert "__ldg(p.alpha" not in text and "__ldg(p.addend" not in text

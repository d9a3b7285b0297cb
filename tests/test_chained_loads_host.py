"""Kernels launched with launch_chained are resident while the kernel ahead
still writes their inputs, and wait for it inside.  Non-coherent loads (__ldg,
or a load through a `const T* __restrict__` parameter, which the compiler may
turn into one) are for memory that nobody writes while a kernel runs; so those
kernels have none.  Read from the sources: no run shows it for sure."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bandwidth_bound_fp8_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _bodies(src):
    """Every function and struct at namespace level: its text, with what precedes the brace."""
    out, depth, start = [], 0, 0
    for m in re.finditer(r"[{};]", src):
        c = m.group()
        if c == "{":
            if re.search(r"namespace\s*\w*\s*$|extern\s*\"C\"\s*$", src[start:m.start()]):
                start = m.end()
                continue
            depth += 1
        elif c == "}":
            depth = max(depth - 1, 0)
            if depth == 0:
                out.append(src[start:m.end()])
                start = m.end()
        elif depth == 0:
            start = m.end()
    return out


@pytest.mark.parametrize("name", ["moeq_rows.cu", "moeq_mx4.cu", "moeq_mx4_plan.cuh", "moeq_mx4_gemm.cu"])
def test_chained_kernels_read_with_plain_loads(name):
    chained = 0
    for body in _bodies(_source(name)):
        kernel = re.search(r"__global__\s.*?\b(\w+_kernel)\(", body, re.S)
        if kernel and "chain();" not in body and "griddepcontrol" not in body and "pdl_wait" not in body:
            continue   # launched plainly: everything ahead has ended before it starts
        chained += bool(kernel)
        what = kernel.group(1) if kernel else body.strip().splitlines()[0]
        assert "__ldg" not in body, what
        if kernel:
            assert not re.search(r"const\s+[\w]+\s*\*\s*__restrict__", body.split("{")[0]), what
    assert chained or name.endswith("cuh")

"""What the library sets once a device (a kernel's attributes): set again on
every other device, and again after a failure; nothing in csrc keeps one
device's, or one failure's, result for the whole process."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bandwidth_bound_fp8_gb300", "csrc")

PROGRAM = """
#include "moeq_once.h"
#include <initializer_list>
int main() {
    static moeq::OncePerDevice once;
    int calls = 0, answer = 7;
    auto set = [&] { ++calls; return answer; };
    if (once.on(0, set) != 7 || calls != 1) return 1;       // a failure is passed on
    if (once.on(0, set) != 7 || calls != 2) return 2;       // and not kept
    answer = 0;
    if (once.on(0, set) != 0 || calls != 3) return 3;
    answer = 9;
    if (once.on(0, set) != 0 || calls != 3) return 4;       // set: not called again
    answer = 0;
    for (int dev : {1, 63, 64, 127})
        if (once.on(dev, set) != 0) return 5;
    if (calls != 7) return 6;                               // each device by itself
    for (int dev : {0, 1, 63, 64, 127})
        if (once.on(dev, set) != 0 || calls != 7) return 7;
    for (int i = 0; i < 3; ++i) once.on(128, set);          // beyond the mask: each time
    return calls == 10 ? 0 : 8;
}
"""


def test_once_per_device(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_no_result_of_a_cuda_call_is_kept_for_the_process():
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, f)) as h:
                assert not re.search(r"static\s+(const\s+)?cudaError_t\s+\w+\s*=", h.read()), f


def test_no_exception_can_leave_the_c_entries():
    """The C entries of the operators on any number of tokens use nothing of C++ that throws."""
    with open(os.path.join(CSRC, "moeq_rows_api.cu")) as h:
        src = re.sub(r"//[^\n]*", "", h.read())
    assert not re.search(r"std::(vector|string|map|mutex|lock_guard|unique_lock|call_once|function)|\bnew\b|\bthrow\b", src)

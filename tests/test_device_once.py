"""What the launchers set once per device (a kernel's limit of shared memory): on every device anew, and again
after a failure."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_refinement_gb300", "csrc")

PROGRAM = r"""
#include "device_once.h"
#include <cstdio>
int main() {
    zs::OncePerDevice once, other;
    int calls = 0, status = 0;
    auto set = [&] { calls++; return status; };
    auto expect = [&](int result, int want, int total, int line) {
        if (result == want && calls == total) return;
        std::printf("line %d: result %d for %d, %d calls for %d\n", line, result, want, calls, total);
        std::exit(1);
    };
    status = 7;  // a failure is told, and not kept
    expect(once.run(0, set), 7, 1, __LINE__);
    status = 0;
    expect(once.run(0, set), 0, 2, __LINE__);
    status = 7;
    expect(once.run(0, set), 0, 2, __LINE__);  // done on this device ...
    expect(once.run(1, set), 7, 3, __LINE__);  // ... and not on the next
    status = 0;
    const int devices[] = {1, 63, 64, 255};
    int total = 3;
    for (int d : devices) expect(once.run(d, set), 0, ++total, __LINE__);
    for (int d : devices) expect(once.run(d, set), 0, total, __LINE__);
    expect(other.run(0, set), 0, ++total, __LINE__);  // another kernel's
    for (int i = 0; i < 2; i++) expect(once.run(256, set), 0, ++total, __LINE__);  // beyond the table: every time
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_once_on_every_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text("#include <cstdlib>\n" + PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_sequence_operators_keep_no_device_state_for_the_process():
    """Their launchers set a kernel's limit by device, never in a static of the process."""
    for name in ("layernorm.cu", "linear.cu", "linear_few.cu", "delta.cu", "delta_bwd.cu", "delta_step.cu", "seq.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "static const cudaError_t" not in text and "cudaFuncSetAttribute" not in text, name

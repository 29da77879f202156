"""Settings that CUDA keeps per device (a kernel's shared-memory limit) are made for every
device that a process uses, and tried again after a failure.  The rule is plain C++ and
runs here without a GPU."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "tern_device.h"
enum Status { kOk = 0, kFailed = 7 };
int main() {
    tern::OncePerDevice once, other;
    int calls = 0;
    Status next = kOk;
    auto set = [&] { ++calls; return next; };
    auto expect = [&](tern::OncePerDevice& o, int device, Status status, int more) {
        const int before = calls;
        const Status got = o(device, set);
        const bool ok = got == status && calls - before == more;
        if (!ok) std::printf("device %d: status %d, %d calls\n", device, got, calls - before);
        return ok;
    };
    bool ok = true;
    ok &= expect(once, 0, kOk, 1) && expect(once, 0, kOk, 0);       // once
    ok &= expect(once, 1, kOk, 1) && expect(once, 63, kOk, 1);      // for each device
    ok &= expect(once, 1, kOk, 0) && expect(once, 0, kOk, 0);
    next = kFailed;
    ok &= expect(once, 2, kFailed, 1) && expect(once, 2, kFailed, 1);   // a failure is not kept
    ok &= expect(once, 0, kOk, 0);
    next = kOk;
    ok &= expect(once, 2, kOk, 1) && expect(once, 2, kOk, 0);
    ok &= expect(once, 64, kOk, 1) && expect(once, 64, kOk, 1) && expect(once, -1, kOk, 1);   // unknown: every time
    ok &= expect(other, 0, kOk, 1);                                     // each kernel for itself
    std::puts(ok ? "ok" : "wrong");
    return ok ? 0 : 1;
}
"""


def test_once_per_device(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs a C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "ternary_bit_weight_gb300", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"

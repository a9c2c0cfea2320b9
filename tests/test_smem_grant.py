"""The shared-memory grants of kernels whose size varies from call to call,
under two host threads: the header's own code, compiled for the host with a
setter in place of the CUDA call."""
import os
import shutil
import subprocess

import pytest

from state_space_sequence_cumsum_gb300 import _build

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem_grant.h"

// The larger request is held inside its setter until the smaller one has been
// answered, or for a third of a second where that one has to wait for it.
int main()
{
    static ssd::SmemGrant grant;
    std::atomic<int> limit{0};
    std::atomic<bool> inside{false}, answered{false};
    std::thread large([&] {
        ssd::raise_smem(grant, 0, 100, [&](int n) {
            limit = n;
            inside = true;
            for (int i = 0; i < 300 && !answered; ++i)
                std::this_thread::sleep_for(std::chrono::milliseconds(1));
            return 0;
        });
    });
    while (!inside)
        std::this_thread::yield();
    std::thread small([&] {
        ssd::raise_smem(grant, 0, 60, [&](int n) { limit = n; return 0; });
        answered = true;
    });
    large.join();
    small.join();
    // what the kernel may take now, and whether a further call for 100 would ask again
    bool asked = false;
    const int e = ssd::raise_smem(grant, 0, 100, [&](int n) { limit = n; asked = true; return 0; });
    // a refused request is passed on and not remembered
    const int refused = ssd::raise_smem(grant, 0, 200, [](int) { return 7; });
    int again = 0;
    ssd::raise_smem(grant, 0, 200, [&](int n) { again = n; return 0; });
    // two devices are apart
    int other = 0;
    ssd::raise_smem(grant, 1, 50, [&](int n) { other = n; return 0; });
    std::printf("%d %d %d %d %d %d\n", (int)limit, (int)asked, e, refused, again, other);
}
"""


def test_a_grant_is_never_lowered(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "grant.cpp", tmp_path / "grant"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", _build.CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([os.fspath(exe)], capture_output=True, text=True, check=True, timeout=60).stdout
    limit, asked, e, refused, again, other = map(int, out.split())
    assert (limit, asked, e) == (100, 0, 0)
    assert (refused, again, other) == (7, 200, 50)

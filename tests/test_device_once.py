"""Setting a kernel up once a device (csrc/lm_device_once.h) from many threads at once, under
the compiler's thread sanitizer: no data race, and nobody goes on before it is set."""
import os
import subprocess
import textwrap

import pytest

from conftest import ROOT

PROGRAM = """
    #include "lm_device_once.h"
    #include <cstdio>
    #include <thread>
    #include <vector>
    int main() {
        static lm::DeviceOnce once;
        std::atomic<int> calls[4] = {}, wrong{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 8; ++t)
            threads.emplace_back([&, t] {
                for (int i = 0; i < 2000; ++i) {
                    const int d = (i + t) % 3;
                    if (!once.run(d, [&] { ++calls[d]; return true; }) || !calls[d]) ++wrong;
                }
            });
        for (auto& t : threads) t.join();
        for (int d = 0; d < 3; ++d)
            if (calls[d] < 1 || calls[d] > 8) ++wrong;
        // one that fails is tried again; no such device
        if (once.run(3, [&] { return false; }) || !once.run(3, [&] { return true; })) ++wrong;
        if (once.run(-1, [] { return true; }) || once.run(64, [] { return true; })) ++wrong;
        return wrong ? 1 : 0;
    }
"""


def test_from_many_threads(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(textwrap.dedent(PROGRAM))
    built = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-I",
                            os.path.join(ROOT, "fp8_gemms_b200", "csrc"), str(src), "-o", str(exe)],
                           capture_output=True, text=True)
    if built.returncode and "tsan" in built.stderr:
        pytest.skip("no thread sanitizer here")
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True)
    if "unexpected memory mapping" in ran.stderr:
        pytest.skip("the thread sanitizer does not run on this kernel")
    assert ran.returncode == 0, ran.stderr

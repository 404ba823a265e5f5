"""What the library keeps of the driver's answers (csrc/sel_per_device.h), in a
host program with answers of its own (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sampling_row_fp32_gb300", "csrc")

PROGRAM = r"""
#include "sel_per_device.h"
#include <cstdio>
#include <thread>
#include <vector>
struct Answer { int a, b; };
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
    static sel::PerDevice<Answer> kept;
    int asked = 0;
    bool works = false;
    auto query = [&](int base) {
        return [&asked, &works, base](Answer& v) { ++asked; v = {base, base + 1}; return works; };
    };
    Answer v{};
    // a failed query is not kept, on any device
    CHECK(!kept.get(0, v, query(10)) && asked == 1);
    CHECK(!kept.get(0, v, query(10)) && asked == 2);
    works = true;
    CHECK(kept.get(0, v, query(10)) && asked == 3 && v.a == 10 && v.b == 11);
    v = {};
    works = false;
    CHECK(kept.get(0, v, query(99)) && asked == 3 && v.a == 10 && v.b == 11);
    // each device has its own
    works = true;
    CHECK(kept.get(1, v, query(20)) && asked == 4 && v.a == 20);
    CHECK(kept.get(63, v, query(30)) && asked == 5 && v.a == 30);
    CHECK(kept.get(0, v, query(99)) && kept.get(1, v, query(99)) && asked == 5 && v.a == 20);
    // ordinals without a place are asked every time
    for (int d : {64, 1000, -1}) {
        int before = asked;
        CHECK(kept.get(d, v, query(40)) && kept.get(d, v, query(50)) && asked == before + 2 && v.a == 50);
    }
    // many threads: one answer, whole
    static sel::PerDevice<Answer> shared;
    std::vector<std::thread> threads;
    std::vector<Answer> got(16);
    for (int i = 0; i < 16; ++i)
        threads.emplace_back([&, i] {
            for (int n = 0; n < 1000; ++n) shared.get(5, got[i], [&](Answer& a) { a = {7, 8}; return true; });
        });
    for (auto& t : threads) t.join();
    for (auto& a : got) CHECK(a.a == 7 && a.b == 8);
    std::puts("ok");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is needed")
def test_only_successful_answers_are_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout

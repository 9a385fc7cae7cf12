"""The record of a kernel's shared-memory allowance: threads that ask for different sizes at once leave the largest
in force, as the record says.  The setter is a stand-in that keeps whatever it was given last."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "page_wise_rank_gb300", "csrc")

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem_limit.h"

int main() {
    using namespace std::chrono_literals;
    static pkv::SmemLimit limit;
    std::atomic<int> in_force{0};
    std::atomic<bool> entered{false}, large_set{false};
    // the smaller request is held inside its setter until the larger one is through, or has had time to be
    std::thread small([&] {
        limit.raise(3, 80, [&](int n) {
            entered = true;
            for (int i = 0; i < 300 && !large_set; ++i) std::this_thread::sleep_for(1ms);
            in_force = n;
            return 0;
        });
    });
    while (!entered) std::this_thread::yield();
    std::thread large([&] {
        limit.raise(3, 150, [&](int n) { in_force = n; return 0; });
        large_set = true;
    });
    small.join();
    large.join();
    int calls = 0;
    auto count = [&](int n) { ++calls; in_force = n; return 0; };
    limit.raise(3, 150, count);                              // as recorded: not set again
    const int kept = in_force;
    limit.raise(3, 100, count);
    const int again = calls;
    const int failed = limit.raise(3, 200, [](int) { return 7; });  // not recorded
    limit.raise(3, 200, count);
    limit.raise(4, 10, count);                               // another device
    std::printf("%d %d %d %d\n", kept, again, failed, calls);
}
"""


def test_threads_asking_for_different_sizes(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=30).stdout.split()
    assert [int(x) for x in got] == [150, 0, 7, 2]

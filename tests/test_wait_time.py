"""How long a bounded wait of the tensor-core kernels has lasted (csrc/wait_time.h),
on the host: its own polls count, the time that another program had the GPU does not."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_kv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "wait_time.h"
using splitzip::WaitTime;
constexpr uint64_t kLimit = 2000000000ull, kSecond = 1000000000ull;

// Polls of `poll` ns until the limit, with the GPU away for `away` ns before every
// `every`-th one; ns of polling.
static uint64_t polled(uint64_t poll, uint64_t away, uint64_t every) {
    uint64_t now = 4000000000ull, own = 0;     // the lower 32 bits wrap on the way
    WaitTime time((uint32_t)now);
    for (uint64_t i = 1; time.waited <= kLimit >> 10; i++) {
        now += poll + (every && i % every == 0 ? away : 0);
        own += poll;
        time.round((uint32_t)now);
    }
    return own;
}

int main() {
    for (uint64_t poll : {32ull, 1000ull, 1024ull, 20000ull, 1000000ull}) {   // shorter than a unit too
        const uint64_t own = polled(poll, 0, 0);
        if (own < kLimit || own > kLimit + 2 * poll + 2048)
            return std::printf("polls of %llu: %llu\n", (unsigned long long)poll, (unsigned long long)own), 1;
    }
    // Once for ten seconds in the middle, or for three every tenth of a second.
    const uint64_t once = polled(20000, 10 * kSecond, 50001), often = polled(20000, 3 * kSecond, 5000);
    if (once < kLimit - kSecond / 10) return std::printf("once: %llu\n", (unsigned long long)once), 1;
    if (often < kLimit / 2) return std::printf("often: %llu\n", (unsigned long long)often), 1;
    return 0;
}
"""


def test_time_away_from_the_gpu_does_not_count(tmp_path):
    src, exe = tmp_path / "wait.cpp", tmp_path / "wait"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


LIMITS = r"""
#include <cstdio>
#include "wait_time.h"
int main() {
    // 2^31 - 256 query rows are at most 2^24 tiles of 128, or of 2 x 64; a tile takes about 1 us.
    for (uint64_t tiles = 0; tiles <= 1ull << 24; tiles += 4099) {
        const uint64_t ns = (uint64_t)splitzip::wait_limit((uint32_t)tiles) << 10;
        if (ns < 1999999000ull + 10000 * tiles || ns > 2000000000ull + 20000 * tiles)
            return std::printf("%llu tiles: %llu ns\n", (unsigned long long)tiles, (unsigned long long)ns), 1;
    }
    return 0;
}
"""


def test_limit_covers_the_longest_valid_wait(tmp_path):
    """A wait of the weights kernel lasts as long as one item: of the most query rows
    that a call may have, 17 seconds."""
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(LIMITS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

"""What a ring of tiles still has in flight when its warps give up (csrc/ring_turns.h), on the host: whichever order
they put their tiles in, the wait is for the last tile of every stage."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_kv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <random>
#include "ring_turns.h"
using splitzip::RingTurns;

// Tiles in any order in which those of a stage are in order, given up after every one of them.
template <int kStages>
static bool any_order(uint32_t seed) {
    std::mt19937 rng(seed);
    constexpr uint32_t kTiles = 23;
    RingTurns<kStages> turns;
    turns.clear();
    bool put[kTiles] = {};
    for (uint32_t done = 0; done < kTiles; done++) {
        uint32_t n;
        do n = rng() % kTiles;
        while (put[n] || (n >= kStages && !put[n - kStages]));
        put[n] = true;
        turns.put(n);
        for (uint32_t s = 0; s < kStages; s++) {
            uint32_t last = kTiles;  // none
            for (uint32_t i = s; i < kTiles && put[i]; i += kStages) last = i;
            if (turns.used(s) != (last < kTiles)) return false;
            if (turns.used(s) && turns.parity(s) != (last / kStages & 1)) return false;
        }
    }
    return true;
}

int main() {
    for (uint32_t seed = 0; seed < 2000; seed++)
        if (!any_order<2>(seed) || !any_order<3>(seed) || !any_order<4>(seed)) return std::printf("seed %u\n", seed), 1;
    // The order of two warps' stores that one number of issued tiles gets wrong: 3 tiles put, 2 of them known.
    RingTurns<3> turns;
    turns.clear();
    turns.put(0), turns.put(2), turns.put(1);
    return turns.used(0) && turns.used(1) && turns.used(2) ? 0 : 2;
}
"""


def test_the_last_tile_of_every_stage_is_waited_for(tmp_path):
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_kernel_keeps_its_tiles_so():
    """The few-row kernel's copies go through RingTurns alone."""
    text = open(os.path.join(CSRC, "paged_rows.cu")).read()
    assert "turns.put(n)" in text and "issued = " not in text

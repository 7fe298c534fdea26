"""The item of work of a group of lanes (csrc/lane_groups.h) on the host, over
the whole range that splitzip_qk_norm_rope accepts: up to 2^31 items of 4 to 16
lanes, so more than 2^32 threads."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_kv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "lane_groups.h"
int main() {
    const uint64_t threads = 128, most = 0x7FFFFFFFull;   // items of one launch
    for (uint64_t lanes = 4; lanes <= 16; lanes *= 2) {
        const uint64_t ctas = (most * lanes + threads - 1) / threads;
        for (uint64_t c = 0; c < ctas; c += c < 1000 || c + 200000 > ctas ? 1 : 9973)
            for (uint64_t t = 0; t < threads; t += lanes / 2) {
                const uint64_t want = (c * threads + t) / lanes;
                const uint64_t got = splitzip::lane_group((uint32_t)c, (uint32_t)t, (uint32_t)threads, (uint32_t)lanes);
                if (got != want) {
                    std::printf("lanes %llu cta %llu thread %llu: item %llu, not %llu\n", (unsigned long long)lanes,
                                (unsigned long long)c, (unsigned long long)t, (unsigned long long)got, (unsigned long long)want);
                    return 1;
                }
            }
    }
    return 0;
}
"""


def test_items_past_two_to_the_32_threads(tmp_path):
    src, exe = tmp_path / "items.cpp", tmp_path / "items"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

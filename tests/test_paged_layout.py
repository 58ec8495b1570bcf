"""The workspace layout of a split chunk on the CPU: the same inline functions that the kernels and the host use, compiled
with the host compiler."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "paged_internal.h"
using namespace kvq;
int main() {
    long odd = 0, bad = 0;
    const int heads[][2] = {{1, 1}, {1, 9}, {3, 3}, {5, 3}, {3, 1}, {8, 5}, {7, 1}, {1, 16}, {9, 1}, {2, 5}, {15, 1}};
    for (int D = 64; D <= 256; D *= 2)
        for (auto& hg : heads)
            for (int sms : {1, 148, 152, 160, 192, 400})
                for (int n_seq = 1; n_seq <= 40; ++n_seq)
                    for (int rows = 1; rows <= 700; rows += rows < 40 ? 1 : 33) {
                        const int H = hg[0], G = hg[1];
                        const int64_t head_rows = (int64_t)rows * H * G;
                        const int splits = prefill_splits((int64_t)rows * G, n_seq, H, D == 256 ? 128 : 256, sms);
                        if (splits < 2) continue;
                        const int64_t pairs = splits * head_rows, at = split_out_at(pairs);
                        odd += pairs & 1;
                        // outputs start behind every (maximum, sum), on 16 bytes, and end inside the workspace
                        bad += at < 2 * pairs || at % 4 || at + pairs * D > paged_prefill_ws_floats(D, head_rows);
                    }
    std::printf("%ld %ld\n", odd, bad);
    return 0;
}
"""


def test_partials_of_a_split_chunk_are_aligned_and_inside(tmp_path):
    cc = shutil.which("g++")
    if not cc:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "layout.cpp", tmp_path / "layout"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-I", os.path.join(ROOT, "quantized_kv_cache_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    odd, bad = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert odd > 1000 and bad == 0

"""Every read of codes that the kernel of many rows makes through registers
(csrc/block_copy.h, k_block_tile of csrc/block_product.hip) lies inside its matrix:
the kernel's loop over the steps replayed by a host program, without a GPU, for
matrices that end anywhere in a block of 128 and rows from 1 to 300 codes."""
import subprocess

from exact_lloyd_means_03_amd import build

SOURCE = r"""
#include <algorithm>
#include <cstdio>
#include "block_copy.h"
using namespace km;

// reads of codes of an M x K matrix that are not inside it
static int64_t outside(bool grad, int64_t M, int64_t K, int64_t splits) {
    const int64_t inner = grad ? M : K, outer = grad ? K : M, ib = (inner + 127) / 128, per = (ib + splits - 1) / splits;
    int64_t bad = 0;
    auto read = [&](int64_t at) { bad += at < 0 || at + 16 > M * K; };
    for (int64_t z = 0; z < splits; ++z) {
        const int64_t s0 = z * per, s1 = std::min(s0 + per, ib);
        if (s0 >= s1) continue;
        for (int64_t o0 = 0; o0 < (outer + 255) / 256 * 256; o0 += 64)
            for (int lane = 0; lane < 64; ++lane)
                for (int i = 0; i < 8; ++i) {
                    const int64_t base = grad ? 0 : std::min(o0, outer - 1) * K;
                    const int64_t wo = tile_matrix_at(grad, K, outer, o0, i, lane), by_step = 128 * (grad ? K : 1);
                    auto bounded = [&](int64_t st) {
                        const int64_t left = std::min<int64_t>(inner - st * 128, 128);
                        int64_t p = base + st * by_step + wo;
                        int n;
                        if (grad) {
                            const int m = i * 16 + (lane >> 2);
                            p -= m < left ? 0 : (m - left + 1) * K;
                            n = (int)std::min<int64_t>(M * K - p, 16);
                        } else {
                            n = (int)left - ((lane & 7) ^ (lane >> 3)) * 16;
                        }
                        read(p - tile_back(n));
                    };
                    auto far = [&](int64_t st) { return std::min(st + kTileStages, s1 - 1); };
                    for (int j = 0; j < kTileStages; ++j) bounded(std::min(s0 + j, s1 - 1));
                    int64_t st = s0;
                    for (; st + 1 + kTileStages < tile_free_end(s1, grad, false); st += 2) {
                        read(base + far(st) * by_step + wo);
                        read(base + far(st + 1) * by_step + wo);
                    }
                    for (; st < s1; ++st) bounded(far(st));
                }
    }
    return bad;
}

int main() {
    int64_t bad = 0;
    auto check = [&](bool grad, int64_t M, int64_t K) {
        for (int64_t splits = 1; splits <= 16; splits *= 2) {
            const int64_t n = outside(grad, M, K, splits);
            if (n) printf("%s M=%lld K=%lld splits=%lld: %lld reads outside\n", grad ? "grad" : "product", (long long)M,
                          (long long)K, (long long)splits, (long long)n);
            bad += n;
        }
    };
    const int64_t widths[] = {1, 2, 3, 5, 7, 9, 14, 15, 16, 17, 31, 63, 65, 130, 257, 300};
    for (int64_t K : widths) {
        for (int64_t M : {16, 17, 100, 127, 128, 129, 255, 300, 2049, 4097}) check(true, M, K);
        for (int64_t M = 513; M <= 1300; M += K < 20 ? 1 : 37) check(true, M, K);
        for (int64_t inner : {16, 17, 127, 128, 129, 641, 655, 769, 1030}) check(false, K, inner);
    }
    return bad != 0;
}
"""


def test_reads_stay_inside(tmp_path):
    src, exe = tmp_path / "reads.cpp", tmp_path / "reads"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:]

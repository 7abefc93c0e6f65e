// Where k_block_tile (block_product.hip) copies codes from, as plain arithmetic that
// a host program can run too (tests/test_block_copy.py checks every read with it).
#pragma once

#include <cstdint>

namespace km {

constexpr int kTileStages = 3;

// 16-byte chunk of row m (of 64 columns) that holds columns 16 c .. 16 c + 15: the
// 32 rows that a transposing read touches spread over all banks.
constexpr int tile_chunk(int c, int m) { return c ^ ((m >> 2 & 1) ^ (m >> 4 & 3)); }

// Copy i of a lane's codes of the matrix, in bytes from the step's first one.  Forward: a
// chunk of row i 8 + lane / 8 behind row o0 (the last one, where there is none).  GRAD: a
// chunk of row i 16 + lane / 4 of the step, columns from o0 on (from 0, where there are none).
constexpr uint32_t tile_matrix_at(bool grad, int64_t K, int64_t outer, int64_t o0, int i, int lane) {
    if (grad) {
        const int64_t row = i * 16 + (lane >> 2), col = o0 + tile_chunk(lane & 3, (int)row) * 16;
        return (uint32_t)(row * K) + (uint32_t)(col < outer ? col : 0);
    }
    const int64_t left = outer - 1 - o0, row = i * 8 + (lane >> 3);
    return (uint32_t)((row < left ? row : left < 0 ? 0 : left) * K) + ((lane & 7) ^ (lane >> 3)) * 16;
}

// Of the steps before s1, those below this one are copied without bounds.  The last one
// ends inside a block of 128; where GRAD copies 16 codes of narrow rows through registers,
// those of the step before it can reach past the end of the matrix (M = 641, K = 1).
constexpr int64_t tile_free_end(int64_t s1, bool grad, bool direct) { return s1 - (grad && !direct ? 2 : 1); }

// A copy of 16 codes of which n are in bounds starts this many bytes lower (load16_in).
constexpr int tile_back(int n) { return n >= 16 ? 0 : 16 - n; }

}  // namespace km

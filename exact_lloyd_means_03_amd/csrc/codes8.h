// Device helpers of the operators that write 8-bit codes (e4m3 with a float32
// scale for each block of 128 columns): reductions over the lanes that hold a
// block, the scale, and the conversion.
#pragma once

#include "rows.h"

namespace km {

template <int V>
struct Int {
    static constexpr int value = V;
};

constexpr int kBlock8 = 128;  // columns (of a matrix: and rows) that share a scale

__host__ __device__ inline int64_t blocks8(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }

// The value of the lane that a DPP control names (every lane takes part).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// f over groups of L lanes (16, 32 or 64, aligned), the result in each of them:
// the lanes at xor 1 and 2, then the mirror images in 8 and in 16, which by then
// hold one value in each half, without LDS; beyond 16 through the wave's shuffle.
template <int L, typename F>
__device__ __forceinline__ uint32_t lane_fold(uint32_t v, F f) {
    v = f(v, dpp<0xb1>(v));
    v = f(v, dpp<0x4e>(v));
    v = f(v, dpp<0x141>(v));
    v = f(v, dpp<0x140>(v));
    if constexpr (L >= 32) v = f(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    if constexpr (L >= 64) v = f(v, (uint32_t)__shfl_xor((int)v, 32, 64));
    return v;
}
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
    return __uint_as_float(lane_fold<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
// Magnitudes as bits: a NaN is larger than all numbers, and stays.
template <int L>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
    return lane_fold<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ uint32_t lane_min(uint32_t v) {
    return lane_fold<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a block of largest magnitude amax (its bits).  At least 2^-100,
// so that its inverse is finite; an infinite or NaN block keeps an infinite or
// NaN scale, and then all its values are NaN.
__device__ __forceinline__ float block_scale(uint32_t amax) {
    const float s = __uint_as_float(amax) * (1.f / 448.f);
    return s < 0x1p-100f ? 0x1p-100f : s;
}

// v / s by the rounded inverse of s: the quotient's remainder, times the inverse,
// corrects the last bit (Markstein), so that codes are those of the division also
// where a quotient lies between two of them; a division costs three times that.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float t = v * inv;
    return fmaf(fmaf(-t, s, v), inv, t);
}

// N values divided by the scale as codes, four in a word.  The quotient is at
// most 448 (1 + 2^-22), which rounds to 448: nothing to clamp.
template <int N>
__device__ __forceinline__ void to_codes(const float (&v)[N], float s, uint32_t (&w)[N / 4]) {
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = quotient(v[4 * i + j], s, inv);
        const int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], p, true);
    }
}

// The codes of a chunk of N elements at p, of which the ones from `skip` on and
// before d are the chunk's own (rows.h: a moved last chunk, a short row).
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ p, int d, int skip, const uint32_t (&w)[N / 4]) {
    typedef uint32_t V __attribute__((ext_vector_type(N / 4)));
    typedef V VU __attribute__((aligned(1)));
    if (skip == 0 && d >= N) {
        V v;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) v[i] = w[i];
        *(VU*)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= skip && i < d) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}
template <>
__device__ __forceinline__ void store_codes<4>(uint8_t* __restrict__ p, int d, int skip, const uint32_t (&w)[1]) {
    typedef uint32_t VU __attribute__((aligned(1)));
    if (skip == 0 && d >= 4) {
        *(VU*)p = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= skip && i < d) p[i] = (uint8_t)(w[0] >> (8 * i));
    }
}

}  // namespace km

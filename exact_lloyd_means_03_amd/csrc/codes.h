// Device helpers of the products with 4-bit weights (codes.hip): decoding of
// a word of eight codes through a 16-entry codebook in registers, the expert
// segment a token tile belongs to, and the 16-bit matrix instructions.
#pragma once

#include "common.h"

namespace km {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A codebook of 16 entries of 16 bits as byte planes: low[0..3] holds the low
// bytes of entries 0-3, 4-7, 8-11, 12-15, high[] the high bytes.
struct Book {
    uint32_t low[4], high[4];
};

// v_perm_b32: selector bytes 0-3 pick from b, 4-7 from a, 0x0c gives 0x00 and
// 0x0d gives 0xff.
__device__ __forceinline__ uint32_t perm(uint32_t a, uint32_t b, uint32_t sel) {
    return __builtin_amdgcn_perm(a, b, sel);
}

// entries: 8 words of two entries each (16 consecutive 16-bit values).
__device__ __forceinline__ Book make_book(const uint32_t (&w)[8]) {
    Book k;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        k.low[i] = perm(w[2 * i + 1], w[2 * i], 0x06040200u);
        k.high[i] = perm(w[2 * i + 1], w[2 * i], 0x07050301u);
    }
    return k;
}

// Four codes, in bits 0-2 of the bytes of sel with bit 3 as the byte masks
// hi8, to the four low and the four high bytes of their entries: entries 0-7
// come from one v_perm of a plane, 8-15 from another, bit 3 of the code
// chooses.
__device__ __forceinline__ void decode4(const Book& k, uint32_t sel, uint32_t hi8, uint32_t* lo, uint32_t* hi) {
    const uint32_t a = perm(k.low[1], k.low[0], sel), b = perm(k.low[3], k.low[2], sel);
    const uint32_t c = perm(k.high[1], k.high[0], sel), d = perm(k.high[3], k.high[2], sel);
    *lo = (b & hi8) | (a & ~hi8);
    *hi = (d & hi8) | (c & ~hi8);
}

// The byte planes of a word's eight codes: the low nibbles of its bytes are
// elements 0-3 (lo[0], hi[0]), the high nibbles elements 4-7.
__device__ __forceinline__ void decode_planes(const Book& k, uint32_t w, uint32_t (&lo)[2], uint32_t (&hi)[2]) {
    const uint32_t e = w & 0x07070707u, o = (w >> 4) & 0x07070707u;
    const uint32_t me = perm(0, 0, ((w >> 3) & 0x01010101u) | 0x0c0c0c0cu);
    const uint32_t mo = perm(0, 0, ((w >> 7) & 0x01010101u) | 0x0c0c0c0cu);
    decode4(k, e, me, &lo[0], &hi[0]);
    decode4(k, o, mo, &lo[1], &hi[1]);
}

// Eight codes of a word to eight 16-bit values in element order.
__device__ __forceinline__ u32x4 decode8(const Book& k, uint32_t w) {
    uint32_t lo[2], hi[2];
    decode_planes(k, w, lo, hi);
    return u32x4{perm(hi[0], lo[0], 0x05010400u), perm(hi[0], lo[0], 0x07030602u), perm(hi[1], lo[1], 0x05010400u),
                 perm(hi[1], lo[1], 0x07030602u)};
}

// 16-bit element types of the products: T selects the matrix instruction.
template <typename T>
struct Half;
template <>
struct Half<_Float16> {
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ uint16_t from(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
    // A scaled weight v = s * entry reaches from 2^-48 to 2^32, float16 from
    // 2^-14 to 2^16.  Weights are kept as 2^13 v where 2^-27 <= |v| < 4 (zeros
    // too), and the others, which a step of the gradient takes in passes of their
    // own, as 2^-16 v where |v| >= 4 (or NaN) and as 2^34 v below: normal
    // numbers, rounded once, in all three windows.
    static constexpr bool kWindows = true;
    typedef _Float16 Scale;  // 2^13 s (exact, or infinite from |s| = 8 on)
    static __device__ __forceinline__ Scale scale(uint16_t s) {
        return __builtin_bit_cast(_Float16, s) * (_Float16)0x1p13f;
    }
    // the eight values of a word times s, each product rounded once: right where
    // none of the codebook's entries strays
    static __device__ __forceinline__ u32x4 decode_scaled(const Book& k, uint32_t w, Scale s) {
        typedef _Float16 H8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(u32x4, __builtin_bit_cast(H8, decode8(k, w)) * (H8)s);
    }
    // How far the products of two entries with s lie from the normal numbers, a
    // half each: 0x7800 or more is outside them (a zero entry or s stays inside,
    // 0 times an infinite s does not).
    typedef uint16_t U2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ U2 strays(uint32_t entries, Scale s) {
        typedef _Float16 H2 __attribute__((ext_vector_type(2)));
        const uint32_t e = entries & 0x7fff7fffu, f = (__builtin_bit_cast(uint16_t, s) & 0x7fffu) * 0x10001u;
        const U2 p = __builtin_bit_cast(U2, __builtin_bit_cast(H2, e) * __builtin_bit_cast(H2, f));
        // 0x0400 where neither factor is zero (a nonzero f is larger): normal numbers, from
        // there to 0x7bff, move to 0 .. 0x77ff, subnormal ones wrap
        const U2 nonzero = __builtin_bit_cast(U2, ((e + 0x7fff7fffu) & 0x80008000u) >> 5);
        return p - __builtin_elementwise_min(nonzero, __builtin_bit_cast(U2, f));
    }
    static __device__ __forceinline__ bool stray(U2 a) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_add_sat(a, (U2)0x0800)) & 0x80008000u;
    }
    // eight entries times s: the weights of a window alone, the others as zeros
    static __device__ __forceinline__ u32x4 one_window(u32x4 x, float s, int window) {
        const float by = window == 0 ? 0x1p13f : window == 1 ? 0x1p-16f : 0x1p34f;
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float v = s * f32((uint16_t)(x[i] >> (16 * e)));  // (exact: 22 bits)
                const int in = !(fabsf(v) < 4.f) ? 1 : v == 0.f || fabsf(v) >= 0x1p-27f ? 0 : 2;
                h[e] = in == window ? from(v * by) : 0;
            }
            r[i] = h[0] | h[1] << 16;
        }
        return r;
    }
};
template <>
struct Half<__bf16> {
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float f32(uint16_t v) { return bf16_to_f32(v); }
    static __device__ __forceinline__ uint16_t from(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
    static constexpr bool kWindows = false;  // float32's range
    typedef float Scale;
    static __device__ __forceinline__ Scale scale(uint16_t s) { return bf16_to_f32(s); }
    // the eight values of a word times s, each product rounded once
    static __device__ __forceinline__ u32x4 decode_scaled(const Book& k, uint32_t w, Scale f) {
        typedef float F2 __attribute__((ext_vector_type(2)));
        typedef __bf16 B2 __attribute__((ext_vector_type(2)));
        uint32_t lo[2], hi[2];
        decode_planes(k, w, lo, hi);
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // bytes to the float32 of elements 2 i and 2 i + 1 (0x0c: zero)
            const uint32_t even = i & 1 ? 0x06020c0cu : 0x04000c0cu, odd = i & 1 ? 0x07030c0cu : 0x05010c0cu;
            const F2 v = {f * __uint_as_float(perm(hi[i / 2], lo[i / 2], even)),
                          f * __uint_as_float(perm(hi[i / 2], lo[i / 2], odd))};
            r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, B2));
        }
        return r;
    }
};

// The segment of token tile y: tiles of TT rows are numbered expert by
// expert, an expert of n rows having ceil(n / TT) of them, and after the last
// expert the rows past offsets[E] (expert E, whose rows become zeros).
// Returns the expert, or -1 if there is no such tile.  Called by whole waves;
// offsets are clamped to [0, S] and made ascending, so that no tile reaches
// outside the rows whatever they hold.
struct Segment {
    int e;
    int64_t p0;
    int n;
};
__device__ __forceinline__ Segment find_segment(const int32_t* __restrict__ offsets, int64_t S, int E, int TT, int y) {
    Segment g{-1, 0, 0};
    if (!offsets) {
        if ((int64_t)y * TT >= S) return g;
        g.e = 0;
        g.p0 = (int64_t)y * TT;
        g.n = S - g.p0 < TT ? (int)(S - g.p0) : TT;
        return g;
    }
    const int lane = threadIdx.x & 63;
    int32_t first = 0;       // tiles of the experts before this round
    int32_t reach = 0;       // the largest offset so far
    for (int e0 = 0; e0 <= E; e0 += 64) {
        const int e = e0 + lane;
        // lane l: rows [a, z) of expert e (the tail after the last one)
        int32_t z = e < E ? offsets[e + 1] : (int32_t)S;
        z = z < 0 ? 0 : z > (int32_t)S ? (int32_t)S : z;
        int32_t m = z;  // running maximum over the lanes
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int32_t t = __shfl_up(m, o, 64);
            if (lane >= o && t > m) m = t;
        }
        if (m < reach) m = reach;
        int32_t a = __shfl_up(m, 1, 64);
        if (lane == 0) a = reach;
        const int32_t tiles = e <= E ? (m - a + TT - 1) / TT : 0;
        int32_t incl = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int32_t t = __shfl_up(incl, o, 64);
            if (lane >= o) incl += t;
        }
        const uint64_t hit = __ballot(first + incl > y);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int32_t before = first + __shfl(incl - tiles, src, 64);
            const int32_t sa = __shfl(a, src, 64), sz = __shfl(m, src, 64);
            // (uniform values: kept in scalar registers)
            const int32_t p0 = __builtin_amdgcn_readfirstlane(sa + (y - before) * TT);
            const int32_t n = __builtin_amdgcn_readfirstlane(sz) - p0;
            g.e = __builtin_amdgcn_readfirstlane(e0 + src);
            g.p0 = p0;
            g.n = n < TT ? n : TT;
            return g;
        }
        first += __shfl(incl, 63, 64);
        reach = __shfl(m, 63, 64);
    }
    return g;
}

// Token tiles a launch must offer for any offsets: every expert and the tail
// may leave one tile partly filled.
inline int64_t segment_tiles(int64_t S, int64_t E, bool offsets, int64_t TT) {
    if (!offsets) return (S + TT - 1) / TT;
    return (S < E + 1 ? S : E + 1) + S / TT;
}

}  // namespace km

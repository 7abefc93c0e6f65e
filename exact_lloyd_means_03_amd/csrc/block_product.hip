// Products of 8-bit rows with 8-bit matrices that have a float32 scale for each
// block of 128 x 128, one matrix per expert, and the gradient of their input.
#include "codes.h"
#include "codes8.h"

namespace km {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// D = A B on a block of 128: 16 x 16 results, lane (r, q) holding 32 codes of
// row r of A and of column r of B (any order of the 128, the same in both).
__device__ __forceinline__ f32x4 mfma8(i32x8 a, i32x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 join8(u32x4 a, u32x4 b) {
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

typedef u32x4 u32x4_byte __attribute__((aligned(1)));

// 16 codes of a row at p, of which p[i], i < n, are in the row (n may be
// negative): the others as zeros.
__device__ __forceinline__ u32x4 load16_end(const uint8_t* __restrict__ p, int n) {
    if (n >= 16) return *(const u32x4_byte*)p;
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < n) v[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    return u32x4{v[0], v[1], v[2], v[3]};
}

// Four consecutive results of a row, the first n (>= 1) of which are in it.
template <typename O>
__device__ __forceinline__ void store_results(O* __restrict__ to, int64_t n, f32x4 v) {
    typedef O V __attribute__((ext_vector_type(4)));
    typedef V VU __attribute__((aligned(sizeof(O))));
    V h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = elem_from<O>(v[e]);
    if (n >= 4) {
        *(VU*)to = h;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) to[e] = h[e];
    }
}

// The row of x that row p of the product is: itself, or by the order (-1: none).
__device__ __forceinline__ int64_t source_row(const int32_t* __restrict__ order, int64_t top, int64_t S, int64_t p) {
    if (!order) return p;
    const int32_t o = order[p];
    return o >= 0 && o < S ? o / (int32_t)top : -1;
}

// Few rows.  out = W x^T on 16 x 16 x 128 instructions, the matrix as A: a block
// takes 16 rows of the matrix and 16 NT tokens, its WK waves every WK-th block
// of 128 columns, whose sums are added in LDS in order.  Codes go from memory to
// operands; GRAD reads the columns of the matrix byte by byte.
template <typename O, int WK, int NT, bool GRAD>
__global__ __launch_bounds__(64 * WK) void k_block_few(const uint8_t* __restrict__ x, const float* __restrict__ xs,
                                                       int64_t S, const uint8_t* __restrict__ codes,
                                                       const float* __restrict__ scales, int E, int64_t M, int64_t K,
                                                       const int32_t* __restrict__ offsets,
                                                       const int32_t* __restrict__ order, int64_t top,
                                                       O* __restrict__ out) {
    constexpr int TT = 16 * NT;
    __shared__ f32x4 s_sum[WK][NT][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const Segment g = find_segment(offsets, S, E, TT, blockIdx.y);
    if (g.e < 0) return;
    // inner: the length summed over; outer: the results of a row
    const int64_t inner = GRAD ? M : K, outer = GRAD ? K : M, ib = blocks8(inner), kb = blocks8(K);
    const int64_t o0 = (int64_t)blockIdx.x * 16, ob = o0 / kBlock8;
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (g.e < E) {
        const uint8_t* wm = codes + (int64_t)g.e * M * K;
        const float* ws = scales + (int64_t)g.e * blocks8(M) * kb;
        const int64_t o = o0 + r < outer ? o0 + r : outer - 1;
        int64_t src[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            src[n] = source_row(order, top, S, g.p0 + (n * 16 + r < g.n ? n * 16 + r : g.n - 1));
        for (int64_t b = w; b < ib; b += WK) {
            const int64_t i0 = b * kBlock8 + q * 32;
            const int left = (int)(inner - i0 < 32 ? inner - i0 : 32);
            u32x4 a[2];
            if constexpr (GRAD) {
                uint32_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j < left) v[j / 4] |= (uint32_t)wm[(i0 + j) * K + o] << (8 * (j % 4));
                a[0] = u32x4{v[0], v[1], v[2], v[3]};
                a[1] = u32x4{v[4], v[5], v[6], v[7]};
            } else {
                a[0] = load16_end(wm + o * K + i0, left);
                a[1] = load16_end(wm + o * K + i0 + 16, left - 16);
            }
            const float sw = GRAD ? ws[b * kb + ob] : ws[ob * kb + b];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint8_t* p = x + src[n] * inner + i0;
                const int have = src[n] < 0 ? 0 : left;
                const u32x4 x0 = load16_end(p, have), x1 = load16_end(p + 16, have - 16);
                const float s = sw * (src[n] < 0 ? 0.f : xs[src[n] * ib + b]);
                const f32x4 d = mfma8(join8(a[0], a[1]), join8(x0, x1), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(s, d[i], acc[n][i]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) s_sum[w][n][lane] = acc[n];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 64; i += 64 * WK) {
        const int n = i >> 6, l = i & 63, tk = n * 16 + (l & 15);
        f32x4 v = s_sum[0][n][l];
#pragma unroll
        for (int o = 1; o < WK; ++o) v += s_sum[o][n][l];
        const int64_t o = o0 + (l >> 4) * 4;
        if (tk < g.n && o < outer) store_results<O>(out + (g.p0 + tk) * outer + o, outer - o, v);
    }
}

size_t block_product_scratch(int64_t, int64_t, int64_t, int64_t) { return 0; }
size_t block_product_grad_scratch(int64_t, int64_t, int64_t, int64_t) { return 0; }

template <typename O, bool GRAD>
static hipError_t block_launch(const BlockArgs& a, hipStream_t s) {
    const int64_t outer = GRAD ? a.K : a.M;
    hipLaunchKernelGGL((k_block_few<O, 8, 1, GRAD>),
                       dim3((unsigned)((outer + 15) / 16), (unsigned)segment_tiles(a.S, a.E, a.offsets, 16)), dim3(512),
                       0, s, (const uint8_t*)a.x, a.x_scales, a.S, (const uint8_t*)a.codes, a.scales, (int)a.E, a.M, a.K,
                       a.offsets, a.order, a.top, (O*)a.out);
    return hipGetLastError();
}

hipError_t launch_block_product(DType ot, bool grad, const BlockArgs& a, void* ws, hipStream_t s) {
    if (a.S == 0) return hipSuccess;
#define KM_GO(O) return grad ? block_launch<O, true>(a, s) : block_launch<O, false>(a, s)
    if (ot == DType::F32) KM_GO(float);
    if (ot == DType::F16) KM_GO(_Float16);
    KM_GO(uint16_t);
#undef KM_GO
}

}  // namespace km

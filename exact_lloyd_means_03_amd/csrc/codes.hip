// Products with 4-bit weights: row codebooks and group scales, one matrix per
// expert (the matrices of github LeanModels/LeanQuant issue #1 "1D k-means":
// every row of weights clustered to 16 values; and of the wpnews.pro "Cache-
// Aware Weight Clustering" post: products straight on codebook and indices).
#include "codes.h"

namespace km {

// labels [M][K] -> tiles (layout in include/kmeans.h).  One thread per 32-bit
// word: 16 bytes per lane and tile, consecutive lanes consecutive words.
__global__ __launch_bounds__(256) void k_pack_codes(const int32_t* __restrict__ labels, int64_t M, int64_t K,
                                                    int64_t KT, int64_t words, uint32_t* __restrict__ codes) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= words) return;
    const int64_t tile = i >> 8;
    const int wd = (int)(i & 255), j = wd & 3, lane = wd >> 2;
    const int64_t m = tile / KT * kCodeRows + (lane & 15);
    const int64_t k0 = tile % KT * kCodeCols + j * 32 + (lane >> 4) * 8;
    uint32_t v = 0;
    if (m < M) {
        for (int e = 0; e < 8; ++e)
            if (k0 + e < K) v |= (uint32_t)(labels[m * K + k0 + e] & 15) << (8 * (e & 3) + 4 * (e >> 2));
    }
    codes[i] = v;
}

hipError_t launch_pack_codes(const int32_t* labels, int64_t M, int64_t K, void* codes, hipStream_t s) {
    const int64_t KT = code_tiles_k(K), words = code_tiles_m(M) * KT * (kCodeTile / 4);
    if (words == 0) return hipSuccess;
    hipLaunchKernelGGL(k_pack_codes, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, labels, M, K, KT, words,
                       (uint32_t*)codes);
    return hipGetLastError();
}

// The codebook of row m of a matrix.
__device__ __forceinline__ Book load_book(const uint16_t* __restrict__ table, int64_t rows, int64_t m) {
    const uint32_t* t = (const uint32_t*)(table + (rows == 1 ? 0 : m) * 16);
    uint32_t w[8];
    if (((uintptr_t)table & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = t[i];
    } else {
        const uint16_t* h = (const uint16_t*)t;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
    return make_book(w);
}

// Eight consecutive 16-bit values at p, those from index n on as zero.
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ p, int n) {
    typedef u32x4 U __attribute__((aligned(2)));
    if (n >= 8) return *(const U*)p;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

// The first n of eight values, the others zero.
__device__ __forceinline__ u32x4 keep8(u32x4 v, int n) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = n >= 2 * i + 2 ? v[i] : n == 2 * i + 1 ? v[i] & 0xffffu : 0u;
    return r;
}

// ---------------------------------------------------------------------------
// Few rows per expert: the codes are streamed once, straight to registers.
//
// out[p][m]: D = W x^T on 16x16x32 matrix instructions, the weights as the
// A operand.  Lane (r, q) of a tile (r < 16 row, q < 4) holds 16 bytes of
// codes, the four words of its row's 32-column steps j, whose eight columns
// q * 8 .. are exactly the eight values it supplies to step j: no exchange
// between lanes.  A block takes one row tile and TT = 16 NT tokens; its waves
// split the columns (tile w, w + W, ...) and add their sums in LDS in wave
// order.  Scales multiply the float32 sum of their group (GS groups in a
// tile), so weights are never rounded after the codebook.
constexpr int kProdWaves = 8;

template <typename T, int NT, int GS>
__global__ __launch_bounds__(64 * kProdWaves) void k_codes_product(
    const uint16_t* __restrict__ x, int64_t S, const char* __restrict__ codes, const uint16_t* __restrict__ table,
    int64_t table_rows, const uint16_t* __restrict__ scales, int64_t group, int64_t groups, int E, int64_t M,
    int64_t K, int64_t MT, int64_t KT, const int32_t* __restrict__ offsets, uint16_t* __restrict__ out) {
    typedef Half<T> H;
    __shared__ f32x4 s_acc[kProdWaves][NT][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const Segment g = find_segment(offsets, S, E, 16 * NT, blockIdx.y);
    if (g.e < 0) return;
    const int64_t mt = blockIdx.x;
    const bool zero = g.e == E;  // rows past the last expert's
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!zero) {
        const char* cm = codes + ((int64_t)g.e * MT + mt) * KT * kCodeTile + lane * 16;
        const uint16_t* xr[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = n * 16 + r < g.n ? n * 16 + r : g.n - 1;  // absent tokens read the last one
            xr[n] = x + (g.p0 + t) * K + q * 8;
        }
        const uint16_t* sc[4];
        if (GS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = mt * 16 + q * 4 + i < M ? mt * 16 + q * 4 + i : M - 1;
                sc[i] = scales + ((int64_t)g.e * M + m) * groups;
            }
        }
        const int64_t mr = mt * 16 + r < M ? mt * 16 + r : M - 1;
        const Book book = load_book(table + (int64_t)g.e * table_rows * 16, table_rows, mr);
        for (int64_t kt = w; kt < KT; kt += kProdWaves) {
            const u32x4 cw = *(const u32x4*)(cm + kt * kCodeTile);
            const int left = (int)(K - kt * kCodeCols < kCodeCols ? K - kt * kCodeCols : kCodeCols);
            u32x4 xv[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xv[n][j] = load8(xr[n] + kt * kCodeCols + j * 32, left == kCodeCols ? 8 : left - j * 32 - q * 8);
            float sv[4][GS ? GS : 1];
            if (GS) {
#pragma unroll
                for (int h = 0; h < GS; ++h) {
                    int64_t gi = GS == 4 ? kt * 4 + h : GS == 2 ? kt * 2 + h : kt * kCodeCols / group;
                    if (gi >= groups) gi = groups - 1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) sv[i][h] = H::f32(sc[i][gi]);
                }
            }
            f32x4 part[NT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 a = decode8(book, cw[j]);
                // columns past the row's end: x is zero there, and so must the weight be (0 * inf is no zero)
                if (left != kCodeCols) a = keep8(a, left - j * 32 - q * 8);
                const bool start = GS && j % (4 / (GS ? GS : 1)) == 0;
                const bool end = GS && (j + 1) % (4 / (GS ? GS : 1)) == 0;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (!GS) {
                        acc[n] = H::mfma(a, xv[n][j], acc[n]);
                    } else {
                        part[n] = H::mfma(a, xv[n][j], start ? f32x4{0.f, 0.f, 0.f, 0.f} : part[n]);
                        if (end) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[n][i] = fmaf(sv[i][j * (GS ? GS : 1) / 4], part[n][i], acc[n][i]);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) s_acc[w][n][lane] = acc[n];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 64; i += 64 * kProdWaves) {
        const int n = i >> 6, l = i & 63;
        f32x4 v = s_acc[0][n][l];
#pragma unroll
        for (int o = 1; o < kProdWaves; ++o) v += s_acc[o][n][l];
        const int t = n * 16 + (l & 15);
        const int64_t m = mt * 16 + (l >> 4) * 4;
        if (t < g.n) {
            uint16_t* to = out + (g.p0 + t) * M + m;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < M) to[e] = H::from(v[e]);
        }
    }
}

size_t codes_product_scratch(int64_t, int64_t, int64_t, int64_t) { return 0; }

// Groups of scales in a tile of 128 columns (1: a group spans whole tiles).
static int groups_per_tile(const CodesArgs& a) {
    if (!a.scales) return 0;
    return a.group == 32 ? 4 : a.group == 64 ? 2 : 1;
}

template <typename T>
static hipError_t product_launch(const CodesArgs& a, hipStream_t s) {
    const int64_t MT = code_tiles_m(a.M), KT = code_tiles_k(a.K);
    const int64_t groups = a.scales ? (a.K + a.group - 1) / a.group : 0;
    const bool few = a.S <= 16 * a.E;
#define KM_GO(NT, GS)                                                                                                \
    hipLaunchKernelGGL((k_codes_product<T, NT, GS>),                                                                 \
                       dim3((unsigned)MT, (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * NT)),                    \
                       dim3(64 * kProdWaves), 0, s, (const uint16_t*)a.x, a.S, (const char*)a.codes,                 \
                       (const uint16_t*)a.table, a.table_rows, (const uint16_t*)a.scales, a.group, groups, (int)a.E, \
                       a.M, a.K, MT, KT, a.offsets, (uint16_t*)a.out)
#define KM_NT(GS)           \
    do {                    \
        if (few) KM_GO(1, GS); \
        else KM_GO(4, GS);  \
    } while (0)
    switch (groups_per_tile(a)) {
        case 0: KM_NT(0); break;
        case 1: KM_NT(1); break;
        case 2: KM_NT(2); break;
        default: KM_NT(4); break;
    }
#undef KM_NT
#undef KM_GO
    return hipGetLastError();
}

hipError_t launch_codes_product(DType xt, const CodesArgs& a, void*, hipStream_t s) {
    if (a.S == 0 || a.M == 0) return hipSuccess;
    return xt == DType::F16 ? product_launch<_Float16>(a, s) : product_launch<__bf16>(a, s);
}

// ---------------------------------------------------------------------------
// The input's gradient: out[p][k] = sum_m g[p][m] W[m][k].
//
// The reduction runs over the rows of the matrix, so the A operand wants
// eight rows of one column per lane where a lane decodes eight columns of one
// row.  A wave decodes 32 rows by 128 columns (two tiles), multiplies by the
// scales, stores them transposed in its own LDS slab and reads operands back.
// Scaled weights are rounded to the 16-bit type there: a scale varies along
// the reduction, so it cannot wait for the float32 sum.
constexpr int kGradWaves = 4, kGradNT = 4, kGradRows = 32;
constexpr int kSlabLd = kGradRows + 8;  // 16-bit elements per column: 80 bytes keep 16-byte reads aligned

template <typename T, int GS>
__global__ __launch_bounds__(64 * kGradWaves) void k_codes_grad(
    const uint16_t* __restrict__ g, int64_t S, const char* __restrict__ codes, const uint16_t* __restrict__ table,
    int64_t table_rows, const uint16_t* __restrict__ scales, int64_t group, int64_t groups, int E, int64_t M,
    int64_t K, int64_t MT, int64_t KT, const int32_t* __restrict__ offsets, uint16_t* __restrict__ out) {
    typedef Half<T> H;
    constexpr int NT = kGradNT, TT = 16 * NT;
    __shared__ __attribute__((aligned(16))) uint16_t s_slab[kGradWaves][kCodeCols * kSlabLd];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const Segment sg = find_segment(offsets, S, E, TT, blockIdx.y);
    if (sg.e < 0) return;
    const int64_t kt = blockIdx.x;
    f32x4 acc[8][NT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[c][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint16_t* slab = s_slab[w];
    if (sg.e < E) {
        const uint16_t* gr[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = n * 16 + r < sg.n ? n * 16 + r : sg.n - 1;
            gr[n] = g + (sg.p0 + t) * M + q * 8;
        }
        const uint16_t* tab = table + (int64_t)sg.e * table_rows * 16;
        for (int64_t m0 = w * kGradRows; m0 < MT * 16; m0 += kGradWaves * kGradRows) {
            u32x4 gv[NT];
            const int64_t left = M - m0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                int have = left >= kGradRows ? 8 : (int)left - q * 8;
                gv[n] = load8(gr[n] + m0, have < 0 ? 0 : have);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t m = m0 + h * 16 + r;
                const bool row = m < M;
                const int64_t mc = row ? m : M - 1;
                const Book book = load_book(tab, table_rows, mc);
                u32x4 cw = u32x4{0, 0, 0, 0};
                if (m0 / 16 + h < MT)
                    cw = *(const u32x4*)(codes + (((int64_t)sg.e * MT + m0 / 16 + h) * KT + kt) * kCodeTile + lane * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u32x4 a = decode8(book, cw[j]);
                    float sv = 1.f;
                    if (GS) {
                        int64_t gi = GS == 1 ? kt * kCodeCols / group : kt * GS + j * GS / 4;
                        if (gi >= groups) gi = groups - 1;
                        sv = H::f32(scales[((int64_t)sg.e * M + mc) * groups + gi]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint16_t v = (uint16_t)(a[e / 2] >> (16 * (e & 1)));
                        if (GS) v = H::from(sv * H::f32(v));
                        slab[(j * 32 + q * 8 + e) * kSlabLd + h * 16 + r] = row ? v : (uint16_t)0;
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const u32x4 a = *(const u32x4*)(slab + (c * 16 + r) * kSlabLd + q * 8);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[c][n] = H::mfma(a, gv[n], acc[c][n]);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
    // add the waves' sums in wave order, 16 columns at a time
    f32x4* s_part = (f32x4*)&s_slab[0][0];  // [kGradWaves][NT][64]
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) s_part[(w * NT + n) * 64 + lane] = acc[c][n];
        __syncthreads();
        const int n = w, l = lane;  // NT == kGradWaves: a wave per token tile
        f32x4 v = s_part[n * 64 + l];
#pragma unroll
        for (int o = 1; o < kGradWaves; ++o) v += s_part[(o * NT + n) * 64 + l];
        const int t = n * 16 + r;
        const int64_t k = kt * kCodeCols + c * 16 + q * 4;
        if (t < sg.n) {
            uint16_t* to = out + (sg.p0 + t) * K + k;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < K) to[e] = H::from(v[e]);
        }
    }
}
static_assert(kGradNT == kGradWaves, "the epilogue gives each wave a token tile");
static_assert(sizeof(f32x4) * kGradWaves * kGradNT * 64 <= sizeof(uint16_t) * kGradWaves * kCodeCols * kSlabLd,
              "the partial sums reuse the slabs");

size_t codes_product_grad_scratch(int64_t, int64_t, int64_t, int64_t) { return 0; }

template <typename T>
static hipError_t grad_launch(const CodesArgs& a, hipStream_t s) {
    const int64_t MT = code_tiles_m(a.M), KT = code_tiles_k(a.K);
    const int64_t groups = a.scales ? (a.K + a.group - 1) / a.group : 0;
#define KM_GO(GS)                                                                                                    \
    hipLaunchKernelGGL((k_codes_grad<T, GS>),                                                                        \
                       dim3((unsigned)KT, (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * kGradNT)),               \
                       dim3(64 * kGradWaves), 0, s, (const uint16_t*)a.x, a.S, (const char*)a.codes,                 \
                       (const uint16_t*)a.table, a.table_rows, (const uint16_t*)a.scales, a.group, groups, (int)a.E, \
                       a.M, a.K, MT, KT, a.offsets, (uint16_t*)a.out)
    switch (groups_per_tile(a)) {
        case 0: KM_GO(0); break;
        case 1: KM_GO(1); break;
        case 2: KM_GO(2); break;
        default: KM_GO(4); break;
    }
#undef KM_GO
    return hipGetLastError();
}

hipError_t launch_codes_product_grad(DType xt, const CodesArgs& a, void*, hipStream_t s) {
    if (a.S == 0 || a.K == 0) return hipSuccess;
    return xt == DType::F16 ? grad_launch<_Float16>(a, s) : grad_launch<__bf16>(a, s);
}

}  // namespace km

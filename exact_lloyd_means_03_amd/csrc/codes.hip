// Products with 4-bit weights: row codebooks and group scales, one matrix per
// expert (the matrices of github LeanModels/LeanQuant issue #1 "1D k-means":
// every row of weights clustered to 16 values; and of the wpnews.pro "Cache-
// Aware Weight Clustering" post: products straight on codebook and indices).
#include "codes.h"
#include "rows.h"

namespace km {

// labels [M][K] -> tiles (layout in include/kmeans.h).  One thread per 32-bit
// word: 16 bytes per lane and tile, consecutive lanes consecutive words.  Done
// once for a matrix: 4096 x 4096 in 36 us, 2.1 TB/s; eight single loads with a
// bound check each are what it waits for.
__global__ __launch_bounds__(256) void k_pack_codes(const int32_t* __restrict__ labels, int64_t M, int64_t K,
                                                    int64_t KT, int64_t words, uint32_t* __restrict__ codes,
                                                    int64_t block0) {
    const int64_t i = (block0 + blockIdx.x) * 256 + threadIdx.x;
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
    in_launches((words + 255) / 256, [&](int64_t b0, unsigned n) {
        hipLaunchKernelGGL(k_pack_codes, dim3(n), dim3(256), 0, s, labels, M, K, KT, words, (uint32_t*)codes, b0);
    });
    return hipGetLastError();
}

template <bool V>
struct Tag {
    static constexpr bool value = V;
};

// The codebook of row m of a matrix: 16 consecutive values, as two vectors.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
__device__ __forceinline__ void fetch_book(const uint16_t* __restrict__ table, int64_t rows, int64_t m, u32x4* a,
                                           u32x4* b) {
    const u32x4_any* t = (const u32x4_any*)(table + (rows == 1 ? 0 : m) * 16);
    *a = t[0];
    *b = t[1];
}
__device__ __forceinline__ Book make_book(u32x4 a, u32x4 b) {
    const uint32_t w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return make_book(w);
}
__device__ __forceinline__ Book load_book(const uint16_t* __restrict__ table, int64_t rows, int64_t m) {
    u32x4 a, b;
    fetch_book(table, rows, m, &a, &b);
    return make_book(a, b);
}

// Eight consecutive 16-bit values of a row.
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ p) { return *(const u32x4_any*)p; }

// The same where only p[i], i < n, are in the row (n may be negative, but
// p[n - 1] is the row's last element): the others as zero.
__device__ __forceinline__ u32x4 load8_end(const uint16_t* __restrict__ p, int n) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint16_t e = p[i < n ? i : n - 1];
        v[i] = i < n ? e : 0u;
    }
    return u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

// The first n of eight values, the others zero.
__device__ __forceinline__ u32x4 keep8(u32x4 v, int n) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = n >= 2 * i + 2 ? v[i] : n == 2 * i + 1 ? v[i] & 0xffffu : 0u;
    return r;
}

// Four consecutive results, the first n (>= 1) of which are in the row.
template <typename T>
__device__ __forceinline__ void store4(uint16_t* __restrict__ to, int64_t n, f32x4 v) {
    typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
    typedef u16x4 u16x4_any __attribute__((aligned(2)));
    u16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = Half<T>::from(v[e]);
    if (n >= 4) {
        *(u16x4_any*)to = h;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) to[e] = h[e];
    }
}

// ---------------------------------------------------------------------------
// The product.
//
// out[p][m]: D = W x^T on 16x16x32 matrix instructions, the weights as the
// A operand.  Lane (r, q) of a tile (r < 16 row, q < 4) holds 16 bytes of
// codes, the four words of its row's 32-column steps j, whose eight columns
// q * 8 .. are exactly the eight values it supplies to step j: the codes go
// from memory to operands in registers, without LDS or an exchange between
// lanes.  Scales multiply the float32 sum of their group (GS groups in a
// tile), so weights are never rounded after the codebook.
//
// A block takes 16 R WR rows of the matrix and 16 NT tokens, a wave R row
// tiles and one of WK parts of the columns.  The columns go by in chunks of
// WK * U tiles, of which a wave has U, all requested a chunk ahead.  A weight
// is decoded (25 instructions for eight) for 16 NT tokens, a token is read
// from LDS for 16 R rows: large blocks where there is enough work to fill the
// device with them, small ones elsewhere (launch rule below).  WK = 1
// exchanges no sums; WK > 1 makes more waves where there are few row tiles,
// and the parts are added in LDS in their order.
//
// X: how tokens come to the operands.  kXDirect: a chunk's tokens go to LDS by
// direct loads of whole lines (the operand layout, 16 bytes from each of 16
// rows, would cost a cache look-up per lane), 16-byte chunks XOR-swizzled by
// the token against bank conflicts.  kXCopy: the same through registers, for
// rows that do not start at 16-byte boundaries.  kXNone: operands straight
// from memory, for one token (broadcasts).
//
// One row by 4096 x 4096 (f16, groups of 128): 6.4 us, a block's chain of
// loads; 64 rows over 16 experts of 4096 x 2048: 24 us for 73 MB (3.0 TB/s),
// vector instructions (decoding) issue 74% of the time; 4096 rows over 8
// experts of 4096 x 4096: 201 us in a stream of calls (684 TFLOP/s; the first
// hundred launches on an idle device 221 us), matrix cores 37%, vector instructions 61% and LDS reads 20% of the cycles.
// 1155 blocks on 512 places (252 registers, 66 KB of LDS) make three rounds, the
// last a quarter full, and an eighth of the token tiles is padding; with experts
// of equal size, two full rounds, it takes 168-172 us.
enum { kXNone, kXDirect, kXCopy };

template <int WR, int WK, int U, int R, int NT, int GS, int X>
struct ProductLds {
    static constexpr int TILE = 16 * NT * kCodeCols * 2;            // x of one tile
    static constexpr int XB = X != kXNone ? 2 * WK * U * TILE : 0;  // two chunks
    static constexpr int SCALE = GS * 64 * 4;                       // a wave's scales: [4 / R tiles][GS][16 R]
    static constexpr int SUMS = WK > 1 ? WR * WK * R * NT * 64 * 16 : 0;
    static constexpr int LOOP = XB + WR * WK * SCALE;
    static constexpr int BYTES = LOOP > SUMS ? LOOP : SUMS;
};

template <typename T, int WR, int WK, int U, int R, int NT, int GS, int X>
__global__ __launch_bounds__(64 * WR * WK) void k_codes_product(
    const uint16_t* __restrict__ x, int64_t S, const char* __restrict__ codes, const uint16_t* __restrict__ table,
    int64_t table_rows, const uint16_t* __restrict__ scales, int64_t group, int64_t groups, int E, int64_t M,
    int64_t K, int64_t MT, int64_t KT, const int32_t* __restrict__ offsets, uint16_t* __restrict__ out) {
    typedef Half<T> H;
    typedef ProductLds<WR, WK, U, R, NT, GS, X> L;
    constexpr bool XLDS = X != kXNone;
    constexpr int TT = 16 * NT, ROW = kCodeCols * 2, NG = GS ? GS : 1, W = WR * WK, CH = WK * U;
    static_assert(U * R <= 4, "16 R lanes load a tile's scales");
    extern __shared__ __attribute__((aligned(16))) char s_mem[];  // x, scales; then the sums
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = w / WK, wk = w % WK, r = lane & 15, q = lane >> 4;
    float* s_scale = (float*)(s_mem + L::XB + w * L::SCALE);  // [4 / R][NG][16 R]
    const Segment g = find_segment(offsets, S, E, TT, blockIdx.y);
    if (g.e < 0) return;
    const int64_t mt = ((int64_t)blockIdx.x * WR + wr) * R;  // the wave's first row tile
    f32x4 acc[R][NT];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[a][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (g.e < E) {  // (expert E stands for the rows past the last expert's)
        const int64_t whole = K / kCodeCols;
        const char* xs = (const char*)(x + g.p0 * K);
        const char* cm[R];
        Book book[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const int64_t mc = mt + a < MT ? mt + a : MT - 1, m = mc * 16 + r < M ? mc * 16 + r : M - 1;
            cm[a] = codes + ((int64_t)g.e * MT + mc) * KT * kCodeTile + lane * 16;
            book[a] = load_book(table + (int64_t)g.e * table_rows * 16, table_rows, m);
        }
        const uint16_t* xr[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = n * 16 + r < g.n ? n * 16 + r : g.n - 1;  // absent tokens read the last one
            xr[n] = (const uint16_t*)xs + (int64_t)t * K + q * 8;
        }
        // a wave's part of a chunk: U tiles of codes a row tile; lane l: the scales of row
        // l % (16 R), tile l / (16 R)
        const int64_t ms = mt * 16 + lane % (16 * R) < M ? mt * 16 + lane % (16 * R) : M - 1;
        const uint16_t* srow = GS ? scales + ((int64_t)g.e * M + ms) * groups : nullptr;
        const int stile = lane / (16 * R) < U ? lane / (16 * R) : U - 1;
        struct Part {
            u32x4 cw[R][U];
            uint16_t sc[NG];
        };
        auto fetch = [&](int64_t c0, Part& p) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t kt = c0 + u * WK + wk;
#pragma unroll
                for (int a = 0; a < R; ++a)
                    p.cw[a][u] = *(const u32x4*)(cm[a] + (kt < KT ? kt : KT - 1) * kCodeTile);
            }
            if (GS) {
                const int64_t kt = c0 + stile * WK + wk;
#pragma unroll
                for (int h = 0; h < NG; ++h) {
                    int64_t gi = GS == 1 ? kt * kCodeCols / group : kt * GS + h;
                    if (gi >= groups) gi = groups - 1;
                    p.sc[h] = srow[gi];
                }
            }
        };
        // the block's x of a chunk, in instructions of 1 KB: 4 tokens by 128 columns
        auto fill = [&](int64_t c0, int buf) {
            constexpr int NI = CH * TT / 4;
#pragma unroll
            for (int i = 0; i < (NI + W - 1) / W; ++i) {
                const int id = i * W + w, ti = id / (TT / 4), tk = id % (TT / 4) * 4 + (lane >> 4);
                const int64_t kt = c0 + ti;
                if (id < NI && kt < whole) {
                    const int64_t src = tk < g.n ? tk : g.n - 1;
                    const uint32_t from = (uint32_t)(src * K * 2 + kt * ROW + ((lane & 15) ^ (tk & 15)) * 16);
                    char* to = s_mem + buf * CH * L::TILE + id * 1024;
                    if (X == kXDirect) dma16(xs, from, to);
                    else *(u32x4*)(to + lane * 16) = load8((const uint16_t*)(xs + from));
                }
            }
        };
        // tile kt from its codes and x; `at` is its place among the wave's scales.
        // END: the last tile of a row that is no multiple of 128 columns.
        auto multiply = [&](int64_t kt, const Part& p, int u, const char* xl, auto end_tag) {
            constexpr bool END = decltype(end_tag)::value;
            const int left = (int)(K - kt * kCodeCols);
            u32x4 av[R][4];
#pragma unroll
            for (int a = 0; a < R; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    av[a][j] = decode8(book[a], p.cw[a][u][j]);
                    // columns past the row's end: x is zero there, and so must the weight be (0 * inf is no zero)
                    if (END) av[a][j] = keep8(av[a][j], left - j * 32 - q * 8);
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                u32x4 xv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint16_t* p = xr[n] + kt * kCodeCols + j * 32;
                    if constexpr (END) xv[j] = load8_end(p, left - j * 32 - q * 8);
                    else if constexpr (XLDS) xv[j] = *(const u32x4*)(xl + (n * 16 + r) * ROW + ((j * 4 + q) ^ r) * 16);
                    else xv[j] = load8(p);
                }
                f32x4 part[R];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool start = GS && j % (4 / NG) == 0, end = GS && (j + 1) % (4 / NG) == 0;
#pragma unroll
                    for (int a = 0; a < R; ++a) {
                        if (!GS) acc[a][n] = H::mfma(av[a][j], xv[j], acc[a][n]);
                        else part[a] = H::mfma(av[a][j], xv[j], start ? f32x4{0.f, 0.f, 0.f, 0.f} : part[a]);
                    }
                    if (end) {
#pragma unroll
                        for (int a = 0; a < R; ++a) {
                            const f32x4 sv = *(const f32x4*)&s_scale[(u * NG + j * NG / 4) * 16 * R + a * 16 + q * 4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[a][n][i] = fmaf(sv[i], part[a][i], acc[a][n][i]);
                        }
                    }
                }
            }
        };
        auto keep_scales = [&](const Part& p) {
            if (GS) {
#pragma unroll
                for (int h = 0; h < NG; ++h) s_scale[(lane / (16 * R) * NG + h) * 16 * R + lane % (16 * R)] = H::f32(p.sc[h]);
            }
        };
        Part p[2];
        fetch(0, p[0]);
        if (XLDS) fill(0, 0);
        for (int64_t c0 = 0; c0 < whole; c0 += 2 * CH) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int64_t c = c0 + b * CH;
                if (c >= whole) break;  // (block-uniform)
                if (XLDS) {
                    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // this wave's direct loads, then everybody's
                    __syncthreads();
                }
                if (c + CH < whole) {
                    fetch(c + CH, p[b ^ 1]);
                    if (XLDS) fill(c + CH, b ^ 1);
                }
                keep_scales(p[b]);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t kt = c + u * WK + wk;
                    if (kt < whole)
                        multiply(kt, p[b], u, s_mem + (b * CH + u * WK + wk) * L::TILE, Tag<false>{});
                }
            }
        }
        if (whole < KT && whole % WK == wk) {
            fetch(whole - wk, p[0]);
            keep_scales(p[0]);
            multiply(whole, p[0], 0, nullptr, Tag<true>{});
        }
    }
    auto store = [&](int n, int64_t tile, int l, f32x4 v) {
        const int tk = n * 16 + (l & 15);
        const int64_t m = tile * 16 + (l >> 4) * 4;
        if (tk < g.n && m < M) store4<T>(out + (g.p0 + tk) * M + m, M - m, v);
    };
    if constexpr (WK == 1) {
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int n = 0; n < NT; ++n) store(n, mt + a, lane, acc[a][n]);
    } else {
        __syncthreads();  // x and scales become the waves' sums
        f32x4* sums = (f32x4*)s_mem;  // [WR][WK][R][NT][64]
        constexpr int PER = R * NT * 64;
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int n = 0; n < NT; ++n) sums[((w * R + a) * NT + n) * 64 + lane] = acc[a][n];
        __syncthreads();
        for (int i = threadIdx.x; i < WR * PER; i += 64 * W) {
            const int row = i / PER, rest = i % PER;
            f32x4 v = sums[row * WK * PER + rest];
#pragma unroll
            for (int o = 1; o < WK; ++o) v += sums[(row * WK + o) * PER + rest];
            store(rest / 64 % NT, ((int64_t)blockIdx.x * WR + row) * R + rest / (64 * NT), rest & 63, v);
        }
    }
}

// Groups of scales in a row (a group may be of any length: no sum with it).
static int64_t groups_per_row(const CodesArgs& a) { return a.scales ? (a.K - 1) / a.group + 1 : 0; }

// Groups of scales in a tile of 128 columns (1: a group spans whole tiles).
static int groups_per_tile(const CodesArgs& a) {
    if (!a.scales) return 0;
    return a.group == 32 ? 4 : a.group == 64 ? 2 : 1;
}

// The launch: the largest block that still makes about one block for every
// compute unit, among those whose tokens' tile is at least half full on
// average over the experts.  Measured (bf16, groups of 128, us a call):
//   tokens, matrices   16 x 32  16 x 128  32 x 64  32 x 128  64 x 128  128 x 128
//     64, 4096 x 4096     14.7      23.5     17.0      25.8      33.3       54.8
//    256, 4096 x 4096     49.4      41.1     28.1      28.4      35.1       56.0
//    512, 4096 x 4096     93.7      75.9     53.5      47.7      37.4       57.3
//   1024, 4096 x 4096    176.1     139.2    102.3      93.5      67.0       61.6
//   2048, 4096 x 4096    328.9     259.5    194.2     167.0     130.6       95.2
//     64, 8 of those      29.1      27.9     29.7      31.6      38.3       63.0
//    512, 8 of those      97.4      74.5     54.2      47.6      39.5       63.5
//   2048, 8 of those     354.2     261.2    189.5     164.6     119.6       93.3
// (tokens x rows of a block).  Rows that are no multiple of 8 columns are copied
// through registers and have three of the blocks, which take half again to four
// times as long (K = 4097, us a call; the last column: what the rule takes at
// K = 4096):
//   tokens, matrices   16 x 16  32 x 128  128 x 128   K = 4096
//     16, 4096 x 4097      9.6      33.6       85.4        8.1
//     64, 4096 x 4097     25.6      36.7       93.3       14.1
//    256, 4096 x 4097     93.5      39.6      113.2       26.8
//   1024, 4096 x 4097    391.9     159.6      154.4       59.9
//   2048, 4096 x 4097    780.1     317.0      174.8       86.3
//     64, 8 of those      58.1      42.8       93.6       26.3
//    512, 8 of those     215.4      85.0      120.9       36.3
//   2048, 8 of those     839.6     318.5      176.2       88.2
// (the rule takes the fastest but at 16 to 128 tokens over 8 matrices, where the
// first stays up to 1.4 times the second).
template <typename T>
static hipError_t product_launch(const CodesArgs& a, hipStream_t s) {
    const int64_t MT = code_tiles_m(a.M), KT = code_tiles_k(a.K);
    const int64_t groups = groups_per_row(a);
    const bool aligned = a.K % 8 == 0 && (uintptr_t)a.x % 16 == 0;
    const int64_t live = a.S < a.E ? a.S : a.E;  // experts with tokens, at most
    auto fits = [&](int64_t tokens, int64_t rows) {
        const int64_t blocks = (MT * 16 + rows - 1) / rows * live * ((a.S + live * tokens - 1) / (live * tokens));
        return (tokens == 16 || 2 * a.S > tokens * a.E) && blocks >= 192;
    };
    hipError_t e = hipSuccess;
#define KM_GO(WR, WK, U, R, NT, GS, X)                                                                                 \
    do {                                                                                                              \
        constexpr size_t lds = ProductLds<WR, WK, U, R, NT, GS, X>::BYTES;                                            \
        if (lds > 64 * 1024 &&                                                                                        \
            (e = hipFuncSetAttribute((const void*)k_codes_product<T, WR, WK, U, R, NT, GS, X>,                        \
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)) != hipSuccess)            \
            return e;                                                                                                 \
        hipLaunchKernelGGL((k_codes_product<T, WR, WK, U, R, NT, GS, X>),                                             \
                           dim3((unsigned)((MT + WR * R - 1) / (WR * R)),                                             \
                                (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * NT)),                               \
                           dim3(64 * WR * WK), lds, s, (const uint16_t*)a.x, a.S, (const char*)a.codes,               \
                           (const uint16_t*)a.table, a.table_rows, (const uint16_t*)a.scales, a.group, groups,        \
                           (int)a.E, a.M, a.K, MT, KT, a.offsets, (uint16_t*)a.out);                                  \
    } while (0)
#define KM_PICK(GS)                                                        \
    do {                                                                   \
        if (a.S == 1) KM_GO(1, 8, 4, 1, 1, GS, kXNone);                    \
        else if (!aligned) {                                               \
            if (fits(128, 128)) KM_GO(4, 1, 1, 2, 8, GS, kXCopy);          \
            else if (fits(32, 128)) KM_GO(8, 1, 4, 1, 2, GS, kXCopy);      \
            else KM_GO(1, 8, 1, 1, 1, GS, kXCopy);                         \
        }                                                                  \
        else if (fits(128, 128)) KM_GO(4, 1, 1, 2, 8, GS, kXDirect);       \
        else if (fits(64, 128)) KM_GO(8, 1, 2, 1, 4, GS, kXDirect);        \
        else if (fits(32, 128)) KM_GO(8, 1, 4, 1, 2, GS, kXDirect);        \
        else if (fits(32, 64)) KM_GO(4, 2, 2, 1, 2, GS, kXDirect);         \
        else if (fits(16, 128)) KM_GO(8, 1, 4, 1, 1, GS, kXDirect);        \
        else if (fits(16, 32)) KM_GO(2, 4, 2, 1, 1, GS, kXDirect);         \
        else KM_GO(1, 8, 1, 1, 1, GS, kXDirect);                           \
    } while (0)
    switch (groups_per_tile(a)) {
        case 0: KM_PICK(0); break;
        case 1: KM_PICK(1); break;
        case 2: KM_PICK(2); break;
        default: KM_PICK(4); break;
    }
#undef KM_PICK
#undef KM_GO
    return hipGetLastError();
}

hipError_t launch_codes_product(DType xt, const CodesArgs& a, hipStream_t s) {
    if (a.S == 0 || a.M == 0) return hipSuccess;
    return xt == DType::F16 ? product_launch<_Float16>(a, s) : product_launch<__bf16>(a, s);
}

// ---------------------------------------------------------------------------
// The input's gradient: out[p][k] = sum_m g[p][m] W[m][k].
//
// The reduction runs over the rows of the matrix, so the A operand wants
// eight rows of one column per lane where a lane decodes eight columns of one
// row.  The eight waves of a block decode a step of 64 rows by 128 columns
// together (half a row tile each), multiply by the scales and store it row by
// row in LDS; transposing reads (ds_read_b64_tr_b16: a lane receives one
// column of four rows) then give the operands, for 64 columns by 16 NTW
// tokens a wave.  Everything a step needs from memory, the tokens' rows of g
// and the tiles' codes, codebooks and scales, comes by direct loads to LDS
// whose lanes take consecutive addresses, one step ahead of its decoding.
//
// Scaled weights are rounded to the 16-bit type's precision before the
// product: the scale varies along the reduction, so it cannot wait for the
// float32 sum.  float16 lacks the range of a product of two of its numbers, so
// weights are held there times 2^13, and a step that has any outside 2^-27 .. 4
// takes its weights in three passes, each with a power of two of its own
// (Half<_Float16>, codes.h).  Looking for such weights costs float16 5 to 8% of
// the time (2048 tokens over 8 experts of 4096 x 2048: 98 us, 92 without it);
// where every step has some, the call takes 460 us.
//
// Few tokens: the rows are split over blockIdx.z and the float32 partial sums
// added in order by k_codes_grad_join.
//
// 2048 tokens over 8 experts of 4096 x 2048 (bf16, groups of 64): 95 us in a
// stream of calls, 360 TFLOP/s (105 us for the first hundred launches on an idle
// device); matrix cores 30% of the cycles, vector instructions 42%, waiting at
// the step's barrier and for LDS most of the rest.  A step moves about 200 KB
// through LDS for 4 MFLOP; tokens loaded straight to operands instead (148 us,
// against 106 then) and half the waves a phase apart (125 us) were slower.
constexpr int kGradWaves = 8, kGradRows = 64;

// 16-byte chunk of row m that holds columns 8 c .. 8 c + 7.  The 16 rows that
// store the same chunk land on 16 distinct ones, and the eight rows that half
// a wave reads (m % 16 in 0-3, 8-11 or in 4-7, 12-15), two chunks each, on
// distinct pairs: neither repeats a bank.
__device__ __forceinline__ int slab_chunk(int c, int m) {
    return c ^ (((m & 3) << 1) | ((m >> 3 & 1) << 3) | (m >> 2 & 1));
}

// What a step brings to LDS.  A token's 64 values are 8 chunks of 16 bytes,
// XOR-swizzled by the token so that the 16 tokens of a B operand lie on
// distinct banks.
template <int TT>
struct GradStage {
    char g[TT * kGradRows * 2];
    char codes[kGradRows / 16 * kCodeTile];
    char book[kGradRows * 32];
    uint32_t scale[4][kGradRows];
};

// DIRECT: rows of g and codebooks start at 16-byte boundaries; otherwise they
// are copied through registers.
template <typename T, int NTW, int GS, bool DIRECT>
__global__ __launch_bounds__(64 * kGradWaves) void k_codes_grad(
    const uint16_t* __restrict__ g, int64_t S, const char* __restrict__ codes, const uint16_t* __restrict__ table,
    int64_t table_rows, const uint16_t* __restrict__ scales, int64_t group, int64_t groups, int E, int64_t M,
    int64_t K, int64_t MT, int64_t KT, const int32_t* __restrict__ offsets, int64_t steps_per, uint16_t* __restrict__ out,
    float* __restrict__ part) {
    typedef Half<T> H;
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    constexpr int TT = kGradWaves / 2 * 16 * NTW, ROW = kCodeCols * 2, C = kCodeCols / 32, GROW = kGradRows * 2;
    extern __shared__ __attribute__((aligned(16))) char s_mem[];
    typedef GradStage<TT> Stage;
    Stage* stage = (Stage*)s_mem;                       // [3]
    auto slab = [&](int b) { return s_mem + 3 * sizeof(Stage) + b * (kGradRows * ROW); };
    // does the step of a slab have weights in other windows: a byte a wave
    constexpr bool WIN = GS && H::kWindows;
    auto others = [&](int b) { return (uint8_t*)s_mem + 3 * sizeof(Stage) + 2 * kGradRows * ROW + b * kGradWaves; };
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const Segment sg = find_segment(offsets, S, E, TT, blockIdx.y);
    if (sg.e < 0) return;
    const int64_t kt = blockIdx.x;
    const int kh = w & 1, th = w >> 1;  // the wave's 64 columns and its 16 NTW tokens
    f32x4 acc[C][NTW];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int n = 0; n < NTW; ++n) acc[c][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t all = (M + kGradRows - 1) / kGradRows;
    const int64_t st0 = blockIdx.z * steps_per, st1 = st0 + steps_per < all ? st0 + steps_per : all;
    if (sg.e < E && st0 < st1) {
        const char* gb = (const char*)(g + sg.p0 * M);
        const char* tab = (const char*)(table + (int64_t)sg.e * table_rows * 16);
        const char* ct = codes + ((int64_t)sg.e * MT * KT + kt) * kCodeTile;
        const char* sc = GS ? (const char*)(scales + (int64_t)sg.e * M * groups) : nullptr;
        // step st to a stage: NTW + 2 direct loads a wave
        auto fill = [&](int64_t st, Stage& to) {
            const int64_t m0 = st * kGradRows;
            const bool whole = m0 + kGradRows <= M;
            if (DIRECT && whole) {
#pragma unroll
                for (int i = 0; i < NTW; ++i) {
                    const int t0 = (i * kGradWaves + w) * 8, t = t0 + (lane >> 3);
                    const int64_t src = t < sg.n ? t : sg.n - 1;
                    dma16(gb, (uint32_t)(src * M * 2 + m0 * 2 + ((lane & 7) ^ (t >> 1 & 7)) * 16), to.g + t0 * GROW);
                }
            } else {
                for (int i = threadIdx.x; i < TT * 8; i += 64 * kGradWaves) {
                    const int t = i >> 3, c = i & 7;
                    const int64_t src = t < sg.n ? t : sg.n - 1;
                    const uint16_t* p = (const uint16_t*)gb + src * M + m0 + c * 8;
                    *(u32x4*)(to.g + t * GROW + (c ^ (t >> 1 & 7)) * 16) =
                        whole ? load8(p) : load8_end(p, (int)(M - m0) - c * 8);
                }
            }
            // waves 0-3: the codes of a row tile each; 4, 5: 32 codebooks each; the scales below
            auto codes_of = [&](int i) {
                const int64_t mt = st * (kGradRows / 16) + i;
                dma16(ct + (mt < MT ? mt : MT - 1) * KT * kCodeTile, lane * 16, to.codes + i * kCodeTile);
            };
            if (w < 4) {
                codes_of(w);
            } else if (w < 6) {
                const int row = (w - 4) * 32 + (lane >> 1);
                const int64_t m = m0 + row < M ? m0 + row : M - 1;
                const uint32_t off = (uint32_t)((table_rows == 1 ? 0 : m) * 32 + (lane & 1) * 16);
                if (DIRECT) dma16(tab, off, to.book + (w - 4) * 1024);
                else *(u32x4*)(to.book + (w - 4) * 1024 + lane * 16) = *(const u32x4_any*)(tab + off);
            }
            const int h = w >= 6 ? w - 6 : w;  // waves 6, 7: groups 0, 1; waves 2, 3: groups 2, 3
            if (GS && (w >= 6 || (GS == 4 && (w == 2 || w == 3))) && h < GS) {
                int64_t gi = GS == 1 ? kt * kCodeCols / group : kt * GS + h;
                if (gi >= groups) gi = groups - 1;
                const int64_t row = m0 + lane < M ? lane : M - 1 - m0;
                dma2(sc + m0 * groups * 2, (uint32_t)((row * groups + gi) * 2), to.scale[h]);
            }
        };
        // the wave's half of a row tile of step st, decoded and scaled, to slab b.
        // ONE: the weights of one window alone.  Otherwise all, as if they lay in the
        // first one, and a byte says whether they do: the lanes of a row share its
        // codebook's entries out.
        auto decode = [&](int64_t st, const Stage& from, int b, int window, auto one_tag) {
            constexpr bool ONE = decltype(one_tag)::value;
            const int row = (w >> 1) * 16 + r;
            const uint2 cw = *(const uint2*)(from.codes + (w >> 1) * kCodeTile + lane * 16 + (w & 1) * 8);
            const u32x4* bk = (const u32x4*)(from.book + row * 32);
            const Book book = make_book(bk[0], bk[1]);
            char* to = slab(b) + row * ROW;
            const bool there = row < (int)(M - st * kGradRows);
            bool stray = false;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int jj = (w & 1) * 2 + j;
                const uint32_t c = j ? cw.y : cw.x;
                const uint16_t s = GS ? (uint16_t)from.scale[jj * GS / 4][row] : 0;
                u32x4 a = GS && !ONE ? H::decode_scaled(book, c, H::scale(s)) : decode8(book, c);
                if constexpr (WIN) {
                    if constexpr (ONE) {
                        a = H::one_window(a, H::f32(s), window);
                    } else if (j == 0 || GS == 4) {  // (else both halves have one scale)
                        const char* e = from.book + row * 32 + q * 8;
                        if (GS == 1) {  // (and the waves of a row too)
                            stray = H::stray(H::strays(*(const uint32_t*)(e + (w & 1) * 4), H::scale(s)));
                        } else {
                            const uint2 e2 = *(const uint2*)e;
                            stray |= H::stray(__builtin_elementwise_max(H::strays(e2.x, H::scale(s)),
                                                                        H::strays(e2.y, H::scale(s))));
                        }
                    }
                }
                if (!there) a = u32x4{0, 0, 0, 0};
                *(u32x4*)(to + slab_chunk(jj * 4 + q, r) * 16) = a;
            }
            // (all lanes store the same byte: no branch between decoding and the product)
            if (WIN && !ONE) others(b)[w] = __ballot(stray) != 0;
        };
        // The slab's weights times the tokens.  ADD: a window's sums, brought to
        // the first one's power of two.
        auto multiply = [&](const char* w16, const Stage& from, float by, auto add_tag) {
            constexpr bool ADD = decltype(add_tag)::value;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 gv[NTW];
#pragma unroll
                for (int n = 0; n < NTW; ++n) {
                    const int t = (th * NTW + n) * 16 + r;
                    gv[n] = *(const u32x4*)(from.g + t * GROW + ((h * 4 + q) ^ (t >> 1 & 7)) * 16);
                }
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    // lane (r, q) wants column c * 16 + r of rows h * 32 + q * 8 .. + 8; it
                    // fetches 8 bytes of row r / 4 (+ 4) of those, columns (r % 4) * 4 ..
                    uint32_t a[4];
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int row = q * 8 + f * 4 + (r >> 2), col = kh * 64 + c * 16 + (r & 3) * 4;
                        const char* at = w16 + (h * 32 + row) * ROW + slab_chunk(col >> 3, row & 15) * 16 + (col & 4) * 2;
                        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4*)at);
                        a[2 * f] = __builtin_bit_cast(uint2, t).x;
                        a[2 * f + 1] = __builtin_bit_cast(uint2, t).y;
                    }
#pragma unroll
                    for (int n = 0; n < NTW; ++n) {
                        const u32x4 av = {a[0], a[1], a[2], a[3]};
                        if constexpr (ADD) acc[c][n] += by * H::mfma(av, gv[n], f32x4{0.f, 0.f, 0.f, 0.f});
                        else acc[c][n] = H::mfma(av, gv[n], acc[c][n]);
                    }
                }
            }
        };
        auto landed = [&]() {  // every load of this wave is in LDS, then every wave's
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
            __syncthreads();
        };
        fill(st0, stage[0]);
        landed();
        if (st0 + 1 < st1) fill(st0 + 1, stage[1]);
        decode(st0, stage[0], 0, 0, Tag<false>{});
        landed();
        int cur = 0, nxt = 1, far = 2, buf = 0;
        for (int64_t st = st0; st < st1; ++st) {
            // here slab `buf` holds step st and stage `nxt` step st + 1
            const uint2 seen = WIN ? *(const uint2*)others(buf) : uint2{0, 0};
            if (st + 2 < st1) fill(st + 2, stage[far]);
            if constexpr (WIN) {
                if (__builtin_amdgcn_readfirstlane(seen.x | seen.y)) {  // (block-uniform)
                    // the other windows, then the first one's weights alone for the usual way
                    for (int window = 2; window >= 0; --window) {
                        decode(st, stage[cur], buf, window, Tag<true>{});
                        __syncthreads();
                        if (window) {
                            multiply(slab(buf), stage[cur], window == 1 ? 0x1p29f : 0x1p-21f, Tag<true>{});
                            __syncthreads();
                        }
                    }
                }
            }
            if (st + 1 < st1) decode(st + 1, stage[nxt], buf ^ 1, 0, Tag<false>{});
            multiply(slab(buf), stage[cur], 1.f, Tag<false>{});
            landed();
            const int t = cur;
            cur = nxt;
            nxt = far;
            far = t;
            buf ^= 1;
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t k = kt * kCodeCols + kh * 64 + c * 16 + q * 4;
        if (k >= K) continue;
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
            const int t = (th * NTW + n) * 16 + r;
            if (t >= sg.n) continue;
            if (WIN) acc[c][n] *= 0x1p-13f;  // (exact)
            const int64_t at = (sg.p0 + t) * K + k;
            if (part) {
                float* to = part + blockIdx.z * S * K + at;
                typedef f32x4 f32x4_any __attribute__((aligned(4)));
                if (k + 4 <= K) {
                    *(f32x4_any*)to = acc[c][n];
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (k + e < K) to[e] = acc[c][n][e];
                }
            } else {
                store4<T>(out + at, K - k, acc[c][n]);
            }
        }
    }
}

// out[i] = the sum of nsplit partial sums, in order; four elements a thread
// (n4 of them, then the rest one by one).
template <typename T>
__global__ __launch_bounds__(256) void k_codes_grad_join(const float* __restrict__ part, int64_t n, int nsplit,
                                                         uint16_t* __restrict__ out) {
    typedef f32x4 f32x4_any __attribute__((aligned(4)));
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    if (i + 4 <= n) {
        f32x4 a = *(const f32x4_any*)(part + i);
        for (int s = 1; s < nsplit; ++s) a += *(const f32x4_any*)(part + s * n + i);
        store4<T>(out + i, 4, a);
    } else {
        for (int64_t j = i; j < n; ++j) {
            float a = part[j];
            for (int s = 1; s < nsplit; ++s) a += part[s * n + j];
            out[j] = Half<T>::from(a);
        }
    }
}

// Tokens of a block (64 ntw) and splits of the rows, by the time they take:
// steps of a block one after the other, in rounds of 256 blocks (one for each
// compute unit), and the partial sums' way through memory.  step_us are a first
// kernel's; measured since, from 4096 and 8192 rows by 256 blocks (bf16 and f16,
// groups of 64 and 128): a step of 64, 128, 256 tokens takes 0.93-0.98, 1.06-1.11
// and 1.28-1.36 us, the same ratios within 5%, and 3-14 us come on top.
// us a call, bf16, groups of 128 (64 ntw tokens / splits; the last column: the
// rule's choice):
//   tokens, matrices    64/1   64/4  64/16  128/1  128/4  256/1  256/4   rule
//     16, 4096 x 4096   65.7   22.5   17.5   71.6   24.5   85.7   28.8   16.2
//    256, 4096 x 4096   67.4   35.5   48.8   73.2   31.5   88.1   35.7   30.1
//    512, 4096 x 4096   69.5   59.9   88.9   78.6   55.4   90.8   41.2   38.7
//   1024, 4096 x 4096   93.5  111.0  180.4   80.0  102.2   92.2   72.5   61.0
//   2048, 4096 x 4096  180.3  213.5  400.9  157.2  198.8   94.4  135.9   94.5
//     64, 8 4096 x 2048 67.7   32.7   43.6   77.1   48.7   91.5   57.4   50.4
//    512, 8 4096 x 2048 69.0   38.6   59.2   79.2   53.2   93.4   61.7   47.0
//   2048, 8 4096 x 2048 94.7  115.5  207.3   81.7  107.9   94.7   76.8   94.9
// It misses where two blocks of 64 or 128 tokens share a compute unit, which it
// counts as two rounds, and where experts of equal size fill their tiles, of
// which it expects half a tile more for each (the last three lines).
struct GradShape {
    int ntw;
    int64_t splits;
};
static GradShape grad_shape(int64_t S, int64_t E, int64_t M, int64_t K) {
    const int64_t live = S < E ? S : E, steps = (M + kGradRows - 1) / kGradRows;
    GradShape best{1, 1};
    if (live < 1) return best;
    double least = 1e30;
    const double step_us[3] = {1.07, 1.26, 1.47};
    for (int i = 0; i < 3; ++i) {
        // token tiles: an expert's last one is half full on average
        const int64_t tt = 64 << i, half = S / tt + (live + 1) / 2;
        const int64_t tiles = E == 1 ? (S + tt - 1) / tt : half > live ? half : live;
        const int64_t blocks = code_tiles_k(K) * tiles;
        for (int64_t n = 1; n <= 64 && (n == 1 || steps / n >= 4); n *= 2) {
            const double rounds = (double)((blocks * n + 255) / 256), per = (double)((steps + n - 1) / n);
            double us = rounds * (per * step_us[i] + 5.0);
            if (n > 1) us += 5.0 + (double)(2 * n * S * K) * sizeof(float) / 3.5e6;
            if (us < least) {
                least = us;
                best = {1 << i, n};
            }
        }
    }
    return best;
}

size_t codes_product_grad_scratch(int64_t S, int64_t E, int64_t M, int64_t K) {
    const int64_t n = grad_shape(S, E, M, K).splits;
    return n > 1 ? ((size_t)(n * S * K) * sizeof(float) + 255) & ~(size_t)255 : 0;
}

template <typename T>
static hipError_t grad_launch(const CodesArgs& a, void* ws, hipStream_t s) {
    const int64_t MT = code_tiles_m(a.M), KT = code_tiles_k(a.K);
    const int64_t groups = groups_per_row(a);
    const GradShape shape = grad_shape(a.S, a.E, a.M, a.K);
    const int64_t nsplit = shape.splits, steps = (a.M + kGradRows - 1) / kGradRows;
    const int64_t per = (steps + nsplit - 1) / nsplit;
    float* part = nsplit > 1 ? (float*)ws : nullptr;
    const bool direct = a.M % 8 == 0 && (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.table % 16 == 0;
    hipError_t e = hipSuccess;
#define KM_GO2(NTW, GS, DIR)                                                                                         \
    do {                                                                                                             \
        constexpr int TT = kGradWaves / 2 * 16 * NTW;                                                                \
        const size_t lds = 3 * sizeof(GradStage<TT>) + 2 * kGradRows * kCodeCols * 2 + 2 * kGradWaves;               \
        if ((e = hipFuncSetAttribute((const void*)k_codes_grad<T, NTW, GS, DIR>,                                     \
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)) != hipSuccess)           \
            return e;                                                                                                \
        hipLaunchKernelGGL((k_codes_grad<T, NTW, GS, DIR>),                                                          \
                           dim3((unsigned)KT, (unsigned)segment_tiles(a.S, a.E, a.offsets, TT), (unsigned)nsplit),   \
                           dim3(64 * kGradWaves), lds, s, (const uint16_t*)a.x, a.S, (const char*)a.codes,           \
                           (const uint16_t*)a.table, a.table_rows, (const uint16_t*)a.scales, a.group, groups,       \
                           (int)a.E, a.M, a.K, MT, KT, a.offsets, per, (uint16_t*)a.out, part);                      \
    } while (0)
#define KM_GO(NTW, GS)                       \
    do {                                     \
        if (direct) KM_GO2(NTW, GS, true);   \
        else KM_GO2(NTW, GS, false);         \
    } while (0)
#define KM_NT(GS)                              \
    do {                                       \
        if (shape.ntw == 1) KM_GO(1, GS);      \
        else if (shape.ntw == 2) KM_GO(2, GS); \
        else KM_GO(4, GS);                     \
    } while (0)
    switch (groups_per_tile(a)) {
        case 0: KM_NT(0); break;
        case 1: KM_NT(1); break;
        case 2: KM_NT(2); break;
        default: KM_NT(4); break;
    }
#undef KM_NT
#undef KM_GO
#undef KM_GO2
    e = hipGetLastError();
    if (e != hipSuccess || nsplit < 2) return e;
    const int64_t n = a.S * a.K;
    hipLaunchKernelGGL((k_codes_grad_join<T>), dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, s, part, n,
                       (int)nsplit, (uint16_t*)a.out);
    return hipGetLastError();
}

hipError_t launch_codes_product_grad(DType xt, const CodesArgs& a, void* ws, hipStream_t s) {
    if (a.S == 0 || a.K == 0) return hipSuccess;
    return xt == DType::F16 ? grad_launch<_Float16>(a, ws, s) : grad_launch<__bf16>(a, ws, s);
}

}  // namespace km

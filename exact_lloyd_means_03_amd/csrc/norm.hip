// The root-mean-square norm of rows with the residual's addition, its
// gradients, and 8-bit codes of rows and matrices.
//
// All are bound by memory: a row is read once into registers, reduced over its
// lanes and written.  A thread owns 16-byte chunks of a row (rows.h); the 16
// lanes (float32: 32) that hold a block of 128 columns are neighbours, so a
// block's largest magnitude needs no LDS.
#include "codes8.h"

namespace km {

// Rows of norms: at most 4096 chunks, so that a block of 16 waves holds one in
// registers.
constexpr int kNormChunks = 4096;
bool norm_fits(int64_t d, DType xt) { return d <= (int64_t)kNormChunks * 16 / dtype_bytes(xt); }

// The weights of a chunk: of the rows' type, or float32; p NULL: ones.
template <typename T>
__device__ __forceinline__ void load_weight(const void* __restrict__ p, bool wide, int e0, int d,
                                            float (&w)[RowVec<T>::N]) {
    constexpr int N = RowVec<T>::N;
    if (!p) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 1.f;
    } else if (!wide) {
        const auto v = load_raw<T>((const T*)p + e0, d);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = elem_f32(v[i]);
    } else {
        const float* f = (const float*)p + e0;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const auto v = d >= N ? load_raw<float>(f + j, 4) : d > j ? load_raw<float>(f + j, d - j) : f32x4{};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[j + i] = v[i];
        }
    }
}

// The sum of v over the WPR waves of a row, in every thread of it.  s: WPR
// floats a row; the waves of a row are all of the block's, where WPR > 1.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* s) {
    v = lane_sum<64>(v);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) v += s[i];
    }
    return v;
}

// WPR waves a row, NC chunks a lane: chunk lane + 64 (wave + WPR i).  The row stays in
// registers as the unrounded float32 sum; a wave alone on its row needs no barrier,
// and rows of up to 8 KB have one, but where there are too few rows to fill the
// device with (fewer than 2048: four waves each).  16421 rows of 4096 bf16 with the
// residual to codes: 98 us, 473 MB at 4.8 TB/s; 8192 of 5120 f16 to f16: 62 us, 5.4
// TB/s; 32 rows of 4096: 4.0 us, a load, a barrier and a store.
//   bf16 to codes with the residual, in a graph, us with four waves a row / with one:
//   rows            32        512       1024       2048        4096        8192
//   of 1024   3.4 / 3.8  3.8 / 4.1  4.7 / 4.2  6.9 / 4.8  10.8 / 6.9  18.5 / 12.7
//   of 2048   3.5 / 5.5  4.1 / 5.9  5.5 / 6.4  7.7 / 7.7  13.8 / 13.4 23.4 / 22.5
//   of 4096   4.0 / 8.9  5.0 / 9.7  7.1 / 10.7 13.0 / 15.6 21.1 / 27.1 37.4 / 45.3
// (the rows of 4096 are found in the memory-side cache there)
template <typename T, int WPR, int NC, bool OUT8>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void k_norm(
    const T* __restrict__ x, const T* __restrict__ res, int64_t Tn, int d, int C, const void* __restrict__ weight,
    bool wide, float eps, T* __restrict__ h, T* __restrict__ y, uint8_t* __restrict__ codes, float* __restrict__ scales,
    int nb, int64_t block0) {
    constexpr int N = RowVec<T>::N, LB = kBlock8 / N;  // lanes of a block
    __shared__ float s_sum[WPR];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t t = WPR == 1 ? (block0 + blockIdx.x) * 4 + w : block0 + blockIdx.x;
    if (t >= Tn) return;  // (whole waves; where waves share a row, no block is without one)
    const int c0 = lane + (WPR == 1 ? 0 : 64 * w);
    float a[NC][N];
    float sum = 0.f;
    typename RowVec<T>::V xv[NC], rv[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + 64 * WPR * i, e0 = chunk_at<T>(c, d);
        xv[i] = rv[i] = typename RowVec<T>::V{};
        if (c < C) {
            xv[i] = load_raw<T>(x + t * d + e0, d);
            if (res) rv[i] = load_raw<T>(res + t * d + e0, d);
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + 64 * WPR * i, e0 = chunk_at<T>(c, d), skip = c * N - e0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            a[i][j] = res ? elem_f32(xv[i][j]) + elem_f32(rv[i][j]) : elem_f32(xv[i][j]);
            if (j >= skip) sum = fmaf(a[i][j], a[i][j], sum);
        }
        if (h && c < C) store_f32<T, N>(h + t * d + e0, d, a[i]);
    }
    const float r = 1.f / sqrtf(row_sum<WPR>(sum, s_sum) / (float)d + eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + 64 * WPR * i, e0 = chunk_at<T>(c, d), skip = c * N - e0;
        float wv[N];
        if (c < C) load_weight<T>(weight, wide, e0, d, wv);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            a[i][j] = c < C ? a[i][j] * r * wv[j] : 0.f;
            if (OUT8 && j >= skip && j < d) top = top > magnitude(a[i][j]) ? top : magnitude(a[i][j]);
        }
        if constexpr (OUT8) {
            const float s = block_scale(lane_max<LB>(top));
            uint32_t q[N / 4];
            to_codes<N>(a[i], s, q);
            if (c < C) {
                store_codes<N>(codes + t * d + e0, d, skip, q);
                if (c % LB == 0) scales[t * nb + c / LB] = s;
            }
        } else if (c < C) {
            store_f32<T, N>(y + t * d + e0, d, a[i]);
        }
    }
}

hipError_t launch_norm(DType xt, const void* x, int64_t T, int64_t d, const void* residual, const void* weight, DType wt,
                       float eps, void* h, void* y, void* codes, float* scales, hipStream_t s) {
    if (T == 0) return hipSuccess;
    const int C = row_chunks(d, dtype_bytes(xt));
    const bool wide = wt == DType::F32 && xt != DType::F32;
    const bool few = T < 2048;
#define KM_GO3(TT, WPR, NC, OUT8)                                                                                       \
    in_launches(WPR == 1 ? (T + 3) / 4 : T, [&](int64_t b0, unsigned n) {                                               \
        hipLaunchKernelGGL((k_norm<TT, WPR, NC, OUT8>), dim3(n), dim3(WPR == 1 ? 256 : 64 * WPR), 0, s,                 \
                           (const TT*)x, (const TT*)residual, T, (int)d, C, weight, wide, eps, (TT*)h, (TT*)y,          \
                           (uint8_t*)codes, scales, (int)blocks8(d), b0);                                               \
    }, WPR)
#define KM_GO2(TT, WPR, NC)                     \
    do {                                        \
        if (codes) KM_GO3(TT, WPR, NC, true);   \
        else KM_GO3(TT, WPR, NC, false);        \
    } while (0)
#define KM_GO(TT)                                        \
    do {                                                 \
        if (C <= 64) KM_GO2(TT, 1, 1);                   \
        else if (few && C <= 512) KM_GO2(TT, 4, 2);      \
        else if (C <= 128) KM_GO2(TT, 1, 2);             \
        else if (C <= 256) KM_GO2(TT, 1, 4);             \
        else if (C <= 512) KM_GO2(TT, 1, 8);             \
        else if (C <= 1024) KM_GO2(TT, 4, 4);            \
        else if (C <= 2048) KM_GO2(TT, 4, 8);            \
        else KM_GO2(TT, 16, 4);                          \
    } while (0)
    if (xt == DType::F32) KM_GO(float);
    else if (xt == DType::F16) KM_GO(_Float16);
    else KM_GO(uint16_t);
#undef KM_GO
#undef KM_GO2
#undef KM_GO3
    return hipGetLastError();
}

// The gradients.  A block of WPR waves takes the rows b, b + G, ... of G blocks;
// a lane keeps the weight gradient's sums of its columns in registers and
// leaves them in part[b], which k_norm_grad_fold adds in the order of b.  Both sums
// of a row (h^2 and u h) come from one reading of it.  8192 rows of 4096 bf16 with
// the residual's gradient: 58 us, 268 MB at 4.6 TB/s, of which the fold takes 5 (in a
// graph that repeats it 50); in such a graph 2048 rows of 16384 take 66 us, 4096 of
// them 126 (4.3 TB/s), 2048 of 32768 176 (3.1 TB/s: what is spilled).
template <typename T, int WPR, int NC, bool GW>
__global__ __launch_bounds__(64 * WPR) void k_norm_grad(const T* __restrict__ grad, const T* __restrict__ hx, int64_t Tn,
                                                        int d, int C, const T* __restrict__ gres,
                                                        const void* __restrict__ weight, bool wide, float eps,
                                                        T* __restrict__ gx, float* __restrict__ part) {
    constexpr int N = RowVec<T>::N;
    __shared__ float s_sum[2][2 * WPR];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c0 = lane + 64 * w;
    // four chunks' weights are read again for every row: kept, they would cost registers
    // that the rows need (two rows of 14016 took 34 us).  Blocks of 16 waves have 128
    // registers a lane: with the weight's gradient, four chunks still spill 28 (f16) or 31
    // (bf16) of them, two chunks of bf16 5
    constexpr bool KEEP = NC < 4;
    float wv[KEEP ? NC : 1][N], acc[NC][N];
    auto weights = [&](int i, float (&v)[N]) {
        const int c = c0 + 64 * WPR * i;
        if (c < C) load_weight<T>(weight, wide, chunk_at<T>(c, d), d, v);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c >= C) v[j] = 0.f;
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if constexpr (KEEP) weights(i, wv[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
    }
    const float dd = (float)d;
    int par = 0;
    for (int64_t t = blockIdx.x; t < Tn; t += gridDim.x, par ^= 1) {
        typename RowVec<T>::V gv[NC], hv[NC], rv[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + 64 * WPR * i, e0 = chunk_at<T>(c, d);
            gv[i] = hv[i] = rv[i] = typename RowVec<T>::V{};
            if (c < C) {
                gv[i] = load_raw<T>(grad + t * d + e0, d);
                hv[i] = load_raw<T>(hx + t * d + e0, d);
                if (gres) rv[i] = load_raw<T>(gres + t * d + e0, d);
            }
        }
        float hh = 0.f, uh = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + 64 * WPR * i, skip = c * N - chunk_at<T>(c, d);
            if constexpr (!KEEP) weights(i, wv[0]);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float hj = elem_f32(hv[i][j]), u = elem_f32(gv[i][j]) * wv[KEEP ? i : 0][j];
                if (j >= skip) {
                    hh = fmaf(hj, hj, hh);
                    uh = fmaf(u, hj, uh);
                }
            }
        }
        hh = lane_sum<64>(hh);
        uh = lane_sum<64>(uh);
        if constexpr (WPR > 1) {
            // two rows' sums in turn: the next row's are written behind this one's barrier
            float* s = s_sum[par];
            if (lane == 0) s[2 * w] = hh, s[2 * w + 1] = uh;
            __syncthreads();
            hh = uh = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) hh += s[2 * i], uh += s[2 * i + 1];
        }
        // (r^3 by itself leaves float32 where h is beyond 2^42 or, with eps 0, below 2^-42)
        const float r = 1.f / sqrtf(hh / dd + eps), k = uh / dd * r * r * r;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + 64 * WPR * i, e0 = chunk_at<T>(c, d);
            if (c >= C) continue;
            if constexpr (!KEEP) {
                weights(i, wv[0]);
                asm("" : "+v"(gv[i]), "+v"(hv[i]));  // (converted again, not kept as float32)
            }
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float hj = elem_f32(hv[i][j]), g = elem_f32(gv[i][j]);
                o[j] = fmaf(r, g * wv[KEEP ? i : 0][j], -hj * k);
                if (gres) o[j] += elem_f32(rv[i][j]);
                if (GW) acc[i][j] = fmaf(g, hj * r, acc[i][j]);
            }
            store_f32<T, N>(gx + t * d + e0, d, o);
        }
    }
    if constexpr (GW) {
        float* p = part + (int64_t)blockIdx.x * d;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + 64 * WPR * i, e0 = chunk_at<T>(c, d);
            if (c < C) store_f32<float, N>(p + e0, d, acc[i]);
        }
    }
}

// out[j] = the sum of part[b][j] over b: 64 columns a block, 16 waves take every
// 16th b, then their sums in order.
__global__ __launch_bounds__(1024) void k_norm_grad_fold(const float* __restrict__ part, int G, int d, int wt,
                                                         void* __restrict__ out) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, j = blockIdx.x * 64 + lane;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (j < d) {
        int b = w;
        for (; b + 48 < G; b += 64) {
#pragma unroll
            for (int u = 0; u < 4; ++u) a[u] += part[(int64_t)(b + 16 * u) * d + j];
        }
        for (; b < G; b += 16) a[0] += part[(int64_t)b * d + j];
    }
    s[w][lane] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (w == 0 && j < d) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += s[i][lane];
        if (wt == (int)DType::F32) ((float*)out)[j] = v;
        else if (wt == (int)DType::F16) ((_Float16*)out)[j] = elem_from<_Float16>(v);
        else ((uint16_t*)out)[j] = elem_from<uint16_t>(v);
    }
}

// Blocks of the gradient, by the shapes alone: each leaves a row of float32 sums, so
// more of them cost the fold, and fewer leave too few rows in flight.  us a call
// (bf16, with the residual's gradient; blocks along the top):
//   rows x columns     512    768   1024   2048   4096
//   32768 x 256       64.9          40.7   32.4   39.4
//   16384 x 1024      51.9   40.7   36.7   44.1
//   16384 x 2048             54.8   57.2   64.3
//    8192 x 4096      52.8   56.0   58.5   65.6
//    8192 x 8192     123.8  116.3
// and 4096 x 16384: 256 blocks 124.8, 384 150.6, 512 132.2.
static int64_t norm_grad_blocks(int64_t T, int C) {
    const int64_t most = C <= 64 ? 2048 : C <= 256 ? 1024 : C <= 512 ? 512 : C <= 1024 ? 768 : 256;
    return T < most ? T : most;
}
size_t norm_grad_scratch(int64_t T, int64_t d, DType xt) {
    return ((size_t)norm_grad_blocks(T, row_chunks(d, dtype_bytes(xt))) * d * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_norm_grad(DType xt, const void* grad, const void* h, int64_t T, int64_t d, const void* gres,
                            const void* weight, DType wt, float eps, void* gx, void* gw, void* ws, hipStream_t s) {
    const int C = row_chunks(d, dtype_bytes(xt));
    const bool wide = wt == DType::F32 && xt != DType::F32;
    const int64_t G = norm_grad_blocks(T, C);
    hipError_t e = hipSuccess;
    if (T > 0) {
#define KM_GO3(TT, WPR, NC, GW)                                                                                         \
    hipLaunchKernelGGL((k_norm_grad<TT, WPR, NC, GW>), dim3((unsigned)G), dim3(64 * WPR), 0, s, (const TT*)grad,        \
                       (const TT*)h, T, (int)d, C, (const TT*)gres, weight, wide, eps, (TT*)gx, (float*)ws)
#define KM_GO2(TT, WPR, NC)                  \
    do {                                     \
        if (gw) KM_GO3(TT, WPR, NC, true);   \
        else KM_GO3(TT, WPR, NC, false);     \
    } while (0)
#define KM_GO(TT)                              \
    do {                                       \
        if (C <= 64) KM_GO2(TT, 1, 1);         \
        else if (C <= 256) KM_GO2(TT, 4, 1);   \
        else if (C <= 512) KM_GO2(TT, 4, 2);   \
        else if (C <= 1024) KM_GO2(TT, 4, 4);  \
        else if (C <= 2048) KM_GO2(TT, 16, 2); \
        else KM_GO2(TT, 16, 4);                \
    } while (0)
        if (xt == DType::F32) KM_GO(float);
        else if (xt == DType::F16) KM_GO(_Float16);
        else KM_GO(uint16_t);
#undef KM_GO
#undef KM_GO2
#undef KM_GO3
        e = hipGetLastError();
    }
    if (e != hipSuccess || !gw) return e;
    hipLaunchKernelGGL(k_norm_grad_fold, dim3((unsigned)((d + 63) / 64)), dim3(1024), 0, s, (const float*)ws, (int)G,
                       (int)d, (int)wt, gw);
    return hipGetLastError();
}

// Codes of rows by blocks of 128 columns: a thread a chunk, a row's chunks
// filled up to whole blocks.  2048 rows of 4096 bf16: 7.1 us, 25 MB at 3.5 TB/s, 6.3
// in a graph that repeats it (one chunk a thread: the launch's start and end weigh).
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_rows(const T* __restrict__ x, int64_t rows, int d, uint32_t C,
                                                       uint8_t* __restrict__ codes, float* __restrict__ scales, int nb,
                                                       int64_t block0) {
    constexpr int N = RowVec<T>::N, LB = kBlock8 / N;
    const ItemBase base = item_base(block0, 256, (uint32_t)nb * LB);
    int64_t t;
    int c;
    item_at(base, threadIdx.x, (uint32_t)nb * LB, &t, &c);
    const bool in = t < rows && (uint32_t)c < C;
    const int e0 = chunk_at<T>(c, d), skip = c * N - e0;
    float a[N];
    uint32_t top = 0;
    typename RowVec<T>::V v{};
    if (in) v = load_raw<T>(x + t * d + e0, d);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        a[j] = elem_f32(v[j]);
        if (in && j >= skip) top = top > magnitude(a[j]) ? top : magnitude(a[j]);
    }
    const float s = block_scale(lane_max<LB>(top));
    uint32_t q[N / 4];
    to_codes<N>(a, s, q);
    if (!in) return;
    store_codes<N>(codes + t * d + e0, d, skip, q);
    if (c % LB == 0) scales[t * nb + c / LB] = s;
}

// Codes of matrices by blocks of 128 x 128: a block of threads each, a thread
// the chunks of one column place in every 16th (float32: 8th) row.  Done once for
// matrices that are held: 8 of 4096 x 4096 bf16 79 us, 403 MB at 5.1 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_matrix(const T* __restrict__ x, int64_t M, int d, int C, int64_t mb,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                         int nb, int64_t block0) {
    constexpr int N = RowVec<T>::N, LB = kBlock8 / N, STEP = 256 / LB, R = kBlock8 / STEP;
    __shared__ uint32_t s_top[4];
    const int64_t at = block0 + blockIdx.x, b = at / nb / mb, m0 = at / nb % mb * kBlock8;
    const int c = (int)(at % nb) * LB + threadIdx.x % LB, e0 = chunk_at<T>(c, d), skip = c * N - e0;
    x += (b * M + m0) * d;
    codes += (b * M + m0) * d;
    float a[R][N];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = threadIdx.x / LB + i * STEP;
        typename RowVec<T>::V v{};
        const bool in = m0 + m < M && c < C;
        if (in) v = load_raw<T>(x + (int64_t)m * d + e0, d);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            a[i][j] = elem_f32(v[j]);
            if (in && j >= skip) top = top > magnitude(a[i][j]) ? top : magnitude(a[i][j]);
        }
    }
    top = lane_max<64>(top);
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = top > s_top[i] ? top : s_top[i];
    const float s = block_scale(top);
    if (threadIdx.x == 0) scales[at] = s;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = threadIdx.x / LB + i * STEP;
        if (m0 + m >= M || c >= C) continue;
        uint32_t q[N / 4];
        to_codes<N>(a[i], s, q);
        store_codes<N>(codes + (int64_t)m * d + e0, d, skip, q);
    }
}

hipError_t launch_quantize(DType xt, const void* x, int64_t B, int64_t M, int64_t K, bool matrix, void* codes,
                           float* scales, hipStream_t s) {
    if (B * M == 0) return hipSuccess;
    const int C = row_chunks(K, dtype_bytes(xt)), nb = (int)blocks8(K);
#define KM_GO(TT)                                                                                                        \
    do {                                                                                                                 \
        if (matrix) {                                                                                                    \
            in_launches(B * blocks8(M) * nb, [&](int64_t b0, unsigned n) {                                               \
                hipLaunchKernelGGL((k_quantize_matrix<TT>), dim3(n), dim3(256), 0, s, (const TT*)x, M, (int)K, C,        \
                                   blocks8(M), (uint8_t*)codes, scales, nb, b0);                                         \
            });                                                                                                          \
        } else {                                                                                                         \
            const int64_t items = B * M * nb * (kBlock8 / RowVec<TT>::N);                                                \
            in_launches((items + 255) / 256, [&](int64_t b0, unsigned n) {                                               \
                hipLaunchKernelGGL((k_quantize_rows<TT>), dim3(n), dim3(256), 0, s, (const TT*)x, B * M, (int)K,         \
                                   (uint32_t)C, (uint8_t*)codes, scales, nb, b0);                                        \
            });                                                                                                          \
        }                                                                                                                \
    } while (0)
    if (xt == DType::F32) KM_GO(float);
    else if (xt == DType::F16) KM_GO(_Float16);
    else KM_GO(uint16_t);
#undef KM_GO
    return hipGetLastError();
}

}  // namespace km

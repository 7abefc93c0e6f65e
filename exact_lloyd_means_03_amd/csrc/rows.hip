// Rows moved by label: the lookup of a table's rows, tokens copied to their
// expert's segment, and the rows brought back with weights.
//
// All of them move every input and output row once and do next to no
// arithmetic, so HBM bounds them.  A thread owns one 16-byte chunk of a row
// (rows.h): consecutive lanes take consecutive chunks and, at the end of a
// row, the next row's, so that rows of any width keep whole waves busy.
#include "rows.h"

namespace km {

constexpr int kRowThreads = 256;

// out[i] = scale * table[labels[i]] (a label outside [0, V): zeros).  The
// product is formed in float32 and rounded once.  U chunks per thread: the
// label and then the row are two dependent loads, U of each are in flight (2
// measured the same, 8 slower by a sixth).  49999 rows of 8 KB from 131072:
// 82 us, 410 MB written at 5.0 TB/s; 32 rows of 4 KB: 4 us.
template <typename T, int U, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_lookup(const T* __restrict__ table, int64_t V, int d, uint32_t C,
                                                        const int32_t* __restrict__ labels, int64_t N, int64_t BN,
                                                        float scale, T* __restrict__ out, int64_t block0) {
    constexpr int VN = RowVec<T>::N;
    const ItemBase base = item_base(block0, (int64_t)kRowThreads * U, C);
    int64_t row[U];
    int e0[U];
    int32_t lab[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int c;
        item_at(base, u * kRowThreads + threadIdx.x, C, &row[u], &c);
        e0[u] = chunk_at<T>(c, d);
        lab[u] = row[u] < BN ? labels[row[u]] : -1;
    }
    typename RowVec<T>::V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = typename RowVec<T>::V{};
        if (lab[u] >= 0 && lab[u] < V) {
            const int64_t b = BN == N ? 0 : row[u] / N;
            v[u] = load_raw<T>(table + (b * V + lab[u]) * d + e0[u], d);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (row[u] >= BN) continue;
        float a[VN];
        const float f = lab[u] >= 0 && lab[u] < V ? scale : 0.f;  // (times zeros, where there is no label)
#pragma unroll
        for (int i = 0; i < VN; ++i) a[i] = f * elem_f32(v[u][i]);
        store_f32<T, VN, STREAM>(out + row[u] * d + e0[u], d, a);
    }
}

hipError_t launch_lookup(DType xt, const void* table, int64_t B, int64_t V, int64_t d, const int32_t* labels,
                         int64_t N, float scale, void* out, hipStream_t s) {
    const int64_t BN = B * N;
    if (BN == 0) return hipSuccess;
    const uint32_t C = row_chunks(d, dtype_bytes(xt));
    constexpr int U = 4;
    const int64_t blocks = (BN * C + kRowThreads * U - 1) / (kRowThreads * U);
    const bool stream = stream_out(BN * d * dtype_bytes(xt));
#define KM_GO2(T, ST)                                                                                            \
    in_launches(blocks, [&](int64_t b0, unsigned n) {                                                            \
        hipLaunchKernelGGL((k_lookup<T, U, ST>), dim3(n), dim3(kRowThreads), 0, s, (const T*)table, V, (int)d, C, \
                           labels, N, BN, scale, (T*)out, b0);                                                   \
    })
#define KM_GO(T)                    \
    do {                            \
        if (stream) KM_GO2(T, true); \
        else KM_GO2(T, false);      \
    } while (0)
    if (xt == DType::F32) KM_GO(float);
    else if (xt == DType::F16) KM_GO(_Float16);
    else KM_GO(uint16_t);
#undef KM_GO
#undef KM_GO2
    return hipGetLastError();
}

// rows[slots[t][k]] = x[t]: each token's chunk is read once and stored to its
// `top` places.  The rows past the last slot (p >= *n_rows) become zero and
// their order -1; they are handled by the thread whose token owns index p.
// 16421 tokens of 4 KB to 6 places: 80-90 us, 470 MB at 5.5 TB/s.
template <typename T, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_dispatch(const T* __restrict__ x, int64_t Tn, int d, uint32_t C,
                                                          int top, const int32_t* __restrict__ slots,
                                                          const int32_t* __restrict__ n_rows, T* __restrict__ rows,
                                                          int32_t* __restrict__ order, int64_t block0) {
    const ItemBase base = item_base(block0, kRowThreads, C);
    int64_t t;
    int c;
    item_at(base, threadIdx.x, C, &t, &c);
    if (t >= Tn) return;
    const int e0 = chunk_at<T>(c, d);
    const auto v = load_raw<T>(x + t * d + e0, d);
    const int32_t n = *n_rows;
    for (int k = 0; k < top; ++k) {
        const int64_t p = t * top + k;
        const int32_t sl = slots[p];
        if (sl >= 0) store_raw<T, STREAM>(rows + (int64_t)sl * d + e0, d, v);
        if (p >= n) {
            store_raw<T>(rows + p * d + e0, d, typename RowVec<T>::V{});
            if (c == 0) order[p] = -1;
        }
    }
}

hipError_t launch_dispatch_rows(DType xt, const void* x, int64_t T, int64_t d, int64_t top, const int32_t* slots,
                                const int32_t* n_rows, void* rows, int32_t* order, hipStream_t s) {
    const uint32_t C = row_chunks(d, dtype_bytes(xt));
    const int64_t blocks = (T * C + kRowThreads - 1) / kRowThreads;
    if (blocks == 0) return hipSuccess;
    const bool stream = stream_out(T * top * d * dtype_bytes(xt));
#define KM_GO2(TT, ST)                                                                                             \
    in_launches(blocks, [&](int64_t b0, unsigned n) {                                                              \
        hipLaunchKernelGGL((k_dispatch<TT, ST>), dim3(n), dim3(kRowThreads), 0, s, (const TT*)x, T, (int)d, C,     \
                           (int)top, slots, n_rows, (TT*)rows, order, b0);                                         \
    })
#define KM_GO(TT)                     \
    do {                              \
        if (stream) KM_GO2(TT, true); \
        else KM_GO2(TT, false);       \
    } while (0)
    // a copy: 16-bit types share the instance
    if (xt == DType::F32) KM_GO(uint32_t);
    else KM_GO(uint16_t);
#undef KM_GO
#undef KM_GO2
    return hipGetLastError();
}

// Few choices (dispatch_small): sort and copy in one launch.  One block per
// token.  The slot of choice i is the number of choices of lower experts plus
// the number of earlier choices of its own expert; every block counts that for
// its own `top` choices over all M = T * top labels, which at this size costs
// less than the launches of a sort.  The block after the last token writes the
// offsets.  24 tokens, 2 choices of 8 experts, rows of 8 KB: 5.2 us, bound by
// latency (labels, counts, rows: three trips to memory).
constexpr int kSmallTop = 8;  // choices counted per pass

template <typename T>
__global__ __launch_bounds__(kRowThreads) void k_dispatch_small(const T* __restrict__ x, int64_t Tn, int d, int C,
                                                                int top, const int32_t* __restrict__ experts, int E,
                                                                T* __restrict__ rows, int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ slots,
                                                                int32_t* __restrict__ order) {
    extern __shared__ int32_t s_h[];  // [E] in the offsets' block
    __shared__ int32_t s_cnt[kSmallTop + 1];
    __shared__ int32_t s_wave[kRowThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int M = (int)Tn * top;
    if ((int64_t)blockIdx.x == Tn) {
        for (int j = tid; j < E; j += kRowThreads) s_h[j] = 0;
        __syncthreads();
        for (int i = tid; i < M; i += kRowThreads) {
            const int32_t l = experts[i];
            if ((uint32_t)l < (uint32_t)E) atomicAdd(&s_h[l], 1);
        }
        __syncthreads();
        int32_t carry = 0;
        for (int j0 = 0; j0 < E; j0 += kRowThreads) {
            const int j = j0 + tid;
            const int32_t v = j < E ? s_h[j] : 0;
            int32_t incl = v;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int32_t u = __shfl_up(incl, o, 64);
                if (lane >= o) incl += u;
            }
            if (lane == 63) s_wave[w] = incl;
            __syncthreads();
            int32_t before = carry, all = 0;
            for (int q = 0; q < kRowThreads / 64; ++q) {
                before += q < w ? s_wave[q] : 0;
                all += s_wave[q];
            }
            if (j < E) offsets[j] = before + incl - v;
            carry += all;
            __syncthreads();
        }
        if (tid == 0) offsets[E] = carry;
        return;
    }
    const int t = blockIdx.x;
    for (int k0 = 0; k0 < top; k0 += kSmallTop) {
        const int nk = top - k0 < kSmallTop ? top - k0 : kSmallTop;
        __syncthreads();
        if (tid <= kSmallTop) s_cnt[tid] = 0;
        __syncthreads();
        int32_t mine[kSmallTop], cnt[kSmallTop], valid = 0;
#pragma unroll
        for (int k = 0; k < kSmallTop; ++k) {
            mine[k] = k < nk ? experts[t * top + k0 + k] : -1;
            cnt[k] = 0;
        }
        for (int i = tid; i < M; i += kRowThreads) {
            const int32_t l = experts[i];
            const bool ok = (uint32_t)l < (uint32_t)E;
            valid += ok;
#pragma unroll
            for (int k = 0; k < kSmallTop; ++k)
                cnt[k] += ok && (l < mine[k] || (l == mine[k] && i < t * top + k0 + k));
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
#pragma unroll
            for (int k = 0; k < kSmallTop; ++k) cnt[k] += __shfl_xor(cnt[k], o, 64);
            valid += __shfl_xor(valid, o, 64);
        }
        if (lane == 0) {
            for (int k = 0; k < nk; ++k) atomicAdd(&s_cnt[k], cnt[k]);
            atomicAdd(&s_cnt[kSmallTop], valid);
        }
        __syncthreads();
        const int n = s_cnt[kSmallTop];
        int32_t sl[kSmallTop];
#pragma unroll
        for (int k = 0; k < kSmallTop; ++k) sl[k] = (uint32_t)mine[k] < (uint32_t)E ? s_cnt[k] : -1;
        if (tid == 0) {
#pragma unroll
            for (int k = 0; k < kSmallTop; ++k) {
                if (k >= nk) continue;
                const int p = t * top + k0 + k;
                slots[p] = sl[k];
                if (sl[k] >= 0) order[sl[k]] = p;
                if (p >= n) order[p] = -1;
            }
        }
        for (int c = tid; c < C; c += kRowThreads) {
            const int e0 = chunk_at<T>(c, d);
            const auto v = load_raw<T>(x + (int64_t)t * d + e0, d);
#pragma unroll
            for (int k = 0; k < kSmallTop; ++k) {
                if (k >= nk) continue;
                const int p = t * top + k0 + k;
                if (sl[k] >= 0) store_raw<T>(rows + (int64_t)sl[k] * d + e0, d, v);
                if (p >= n) store_raw<T>(rows + (int64_t)p * d + e0, d, typename RowVec<T>::V{});
            }
        }
    }
}

hipError_t launch_dispatch_small(DType xt, const void* x, int64_t T, int64_t d, int64_t top, const int32_t* experts,
                                 int64_t E, void* rows, int32_t* offsets, int32_t* slots, int32_t* order,
                                 hipStream_t s) {
    const int C = row_chunks(d, dtype_bytes(xt));
    const size_t lds = (size_t)E * sizeof(int32_t);
#define KM_GO(TT)                                                                                                  \
    hipLaunchKernelGGL((k_dispatch_small<TT>), dim3((unsigned)(T + 1)), dim3(kRowThreads), lds, s, (const TT*)x, T, \
                       (int)d, C, (int)top, experts, (int)E, (TT*)rows, offsets, slots, order)
    if (xt == DType::F32) KM_GO(uint32_t);
    else KM_GO(uint16_t);
#undef KM_GO
    return hipGetLastError();
}

// out[t] = sum_k w[t][k] rows[slots[t][k]] (w NULL: all 1), summed in float32
// in the order of k and rounded once; a choice without a slot adds nothing.
// U rows are in flight per thread.  6 x 16421 rows of 4 KB: 93 us, 470 MB at
// 5.0 TB/s.
template <typename T, bool WEIGHTED, int U, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_combine(const T* __restrict__ rows, int64_t Tn, int d, uint32_t C,
                                                         int top, const int32_t* __restrict__ slots,
                                                         const float* __restrict__ w, T* __restrict__ out, int64_t block0) {
    constexpr int VN = RowVec<T>::N;
    const ItemBase base = item_base(block0, kRowThreads, C);
    int64_t t;
    int c;
    item_at(base, threadIdx.x, C, &t, &c);
    if (t >= Tn) return;
    const int e0 = chunk_at<T>(c, d);
    const int64_t S = Tn * top;
    float acc[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) acc[i] = 0.f;
    for (int k0 = 0; k0 < top; k0 += U) {
        int64_t sl[U];
        float wk[U];
        typename RowVec<T>::V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sl[u] = k0 + u < top ? slots[t * top + k0 + u] : -1;
            if (sl[u] >= S) sl[u] = -1;
            wk[u] = WEIGHTED && k0 + u < top ? w[t * top + k0 + u] : 1.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = typename RowVec<T>::V{};
            if (sl[u] >= 0) v[u] = load_raw<T>(rows + sl[u] * d + e0, d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (sl[u] < 0) continue;
#pragma unroll
            for (int i = 0; i < VN; ++i) acc[i] = WEIGHTED ? fmaf(wk[u], elem_f32(v[u][i]), acc[i]) : acc[i] + elem_f32(v[u][i]);
        }
    }
    store_f32<T, VN, STREAM>(out + t * d + e0, d, acc);
}

hipError_t launch_combine(DType xt, const void* rows, int64_t T, int64_t d, int64_t top, const int32_t* slots,
                          const float* w, void* out, hipStream_t s) {
    const uint32_t C = row_chunks(d, dtype_bytes(xt));
    const int64_t blocks = (T * C + kRowThreads - 1) / kRowThreads;
    if (blocks == 0) return hipSuccess;
    const bool stream = stream_out(T * d * dtype_bytes(xt));
#define KM_GO4(TT, WT, U, ST)                                                                                       \
    in_launches(blocks, [&](int64_t b0, unsigned n) {                                                               \
        hipLaunchKernelGGL((k_combine<TT, WT, U, ST>), dim3(n), dim3(kRowThreads), 0, s, (const TT*)rows, T, (int)d, \
                           C, (int)top, slots, w, (TT*)out, b0);                                                    \
    })
#define KM_GO3(TT, WT, U)                     \
    do {                                      \
        if (stream) KM_GO4(TT, WT, U, true);  \
        else KM_GO4(TT, WT, U, false);        \
    } while (0)
#define KM_GO2(TT, WT)                    \
    do {                                  \
        if (top <= 2) KM_GO3(TT, WT, 2);  \
        else if (top <= 4) KM_GO3(TT, WT, 4); \
        else KM_GO3(TT, WT, 8);           \
    } while (0)
#define KM_GO(TT)                \
    do {                         \
        if (w) KM_GO2(TT, true); \
        else KM_GO2(TT, false);  \
    } while (0)
    if (xt == DType::F32) KM_GO(float);
    else if (xt == DType::F16) KM_GO(_Float16);
    else KM_GO(uint16_t);
#undef KM_GO
#undef KM_GO2
#undef KM_GO3
#undef KM_GO4
    return hipGetLastError();
}

// Gradients of the weighted return: grows[slots[t][k]] = w[t][k] gy[t], and
// gw[t][k] = <gy[t], rows[slots[t][k]]> (0 without a slot), the dot in
// float32: each lane sums its chunks in order, then a fixed tree over the
// lanes and waves.  WPT waves per token; gy's chunk is read once for KB
// choices.  Rows past the last slot (order < 0) become zero.  8192 tokens of
// 8 KB, 4 choices: 124 us, 604 MB at 4.9 TB/s.
template <typename T, int WPT, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_combine_grad(const T* __restrict__ gy, const T* __restrict__ rows,
                                                              int64_t Tn, int d, int C, int top,
                                                              const int32_t* __restrict__ slots,
                                                              const int32_t* __restrict__ order,
                                                              const float* __restrict__ w, T* __restrict__ grows,
                                                              float* __restrict__ gw, int64_t block0) {
    constexpr int VN = RowVec<T>::N, KB = 4, NW = kRowThreads / 64;
    __shared__ float s_dot[NW][KB];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t = (block0 + blockIdx.x) * (NW / WPT) + wv / WPT;
    if (WPT < NW && t >= Tn) return;  // (WPT == NW: every block has a token)
    const int64_t S = Tn * top;
    const int64_t tt = t;
    for (int k0 = 0; k0 < top; k0 += KB) {
        int64_t sl[KB];
        float wk[KB], dot[KB];
        bool empty[KB];
#pragma unroll
        for (int u = 0; u < KB; ++u) {
            const bool in = k0 + u < top;
            const int64_t p = tt * top + k0 + u;
            sl[u] = in ? slots[p] : -1;
            if (sl[u] >= S) sl[u] = -1;
            wk[u] = in ? w[p] : 0.f;
            empty[u] = in && order[p] < 0;
            dot[u] = 0.f;
        }
        for (int c = lane + 64 * (wv % WPT); c < C; c += 64 * WPT) {
            const int e0 = chunk_at<T>(c, d);
            const int skip = c * VN - e0;  // elements of an overlapping last chunk already in the one before
            const auto g = load_raw<T>(gy + tt * d + e0, d);
            typename RowVec<T>::V r[KB];
#pragma unroll
            for (int u = 0; u < KB; ++u) {
                r[u] = typename RowVec<T>::V{};
                if (sl[u] >= 0) r[u] = load_raw<T>(rows + sl[u] * d + e0, d);
            }
#pragma unroll
            for (int u = 0; u < KB; ++u) {
                if (sl[u] >= 0) {
                    float a[VN];
#pragma unroll
                    for (int i = 0; i < VN; ++i) {
                        const float gi = elem_f32(g[i]);
                        a[i] = wk[u] * gi;
                        if (i >= skip) dot[u] = fmaf(gi, elem_f32(r[u][i]), dot[u]);
                    }
                    store_f32<T, VN, STREAM>(grows + sl[u] * d + e0, d, a);
                }
                if (empty[u]) store_raw<T>(grows + (tt * top + k0 + u) * d + e0, d, typename RowVec<T>::V{});
            }
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
#pragma unroll
            for (int u = 0; u < KB; ++u) dot[u] += __shfl_xor(dot[u], o, 64);
        }
        if constexpr (WPT == 1) {
#pragma unroll
            for (int u = 0; u < KB; ++u)
                if (lane == u && k0 + u < top) gw[tt * top + k0 + u] = dot[u];
        } else {
            if (lane == 0) {
#pragma unroll
                for (int u = 0; u < KB; ++u) s_dot[wv][u] = dot[u];
            }
            __syncthreads();
            if (threadIdx.x < KB && k0 + (int)threadIdx.x < top) {
                float a = 0.f;
#pragma unroll
                for (int q = 0; q < NW; ++q) a += s_dot[q][threadIdx.x];
                gw[tt * top + k0 + threadIdx.x] = a;
            }
            __syncthreads();
        }
    }
}

hipError_t launch_combine_grad(DType xt, const void* gy, const void* rows, int64_t T, int64_t d, int64_t top,
                               const int32_t* slots, const int32_t* order, const float* w, void* grows, float* gw,
                               hipStream_t s) {
    if (T == 0) return hipSuccess;
    const int C = row_chunks(d, dtype_bytes(xt));
    const bool wide = C > 128;  // two chunks or more a lane: four waves share a token
    const bool stream = stream_out(T * top * d * dtype_bytes(xt));
#define KM_GO3(TT, WPT, ST)                                                                                         \
    in_launches((T * (WPT) + 3) / 4, [&](int64_t b0, unsigned n) {                                                  \
        hipLaunchKernelGGL((k_combine_grad<TT, WPT, ST>), dim3(n), dim3(kRowThreads), 0, s, (const TT*)gy,          \
                           (const TT*)rows, T, (int)d, C, (int)top, slots, order, w, (TT*)grows, gw, b0);           \
    })
#define KM_GO2(TT, WPT)                     \
    do {                                    \
        if (stream) KM_GO3(TT, WPT, true);  \
        else KM_GO3(TT, WPT, false);        \
    } while (0)
#define KM_GO(TT)               \
    do {                        \
        if (wide) KM_GO2(TT, 4); \
        else KM_GO2(TT, 1);     \
    } while (0)
    if (xt == DType::F32) KM_GO(float);
    else if (xt == DType::F16) KM_GO(_Float16);
    else KM_GO(uint16_t);
#undef KM_GO
#undef KM_GO2
#undef KM_GO3
    return hipGetLastError();
}

}  // namespace km

// Stable sorts of labels for the operators that move rows by label.
//
// The sort of a Lloyd fit (sort.hip) has at most 32768 clusters and hands
// out the permutation.  Routing needs the inverse (the place of every
// choice), and a vocabulary has more labels than a counting sort keeps bins
// for.  Both are built here from one counting pass over a digit of at most
// 4097 values (k_digit_hist, the column scan of sort.hip, k_digit_rank):
//   - routing: one pass over the experts, handing out each choice's place;
//   - vocabularies: least significant digit first, in one pass up to 4096
//     labels and else ceil(bits / 12) passes, each stable, so that the last one
//     leaves labels in ascending order and the indices of a label in ascending
//     order.  131072 labels of 17 bits: two passes of 15 us, latency of
//     dependent launches.
// Short label vectors skip the passes: k_count_rank counts, for every label,
// the ones that sort before it.
//
// Every step is a deterministic function of the labels.
#include "common.h"

namespace km {

constexpr int kRankThreads = 512, kRankWaves = kRankThreads / 64;

// Labels per chunk of a pass: whole rounds of the block, at most 256 chunks
// in the job and per problem (the column scan's limit).
int64_t rank_chunk(int64_t B, int64_t N) {
    int64_t ch = 512;
    while (ch < N && B * ((N + ch - 1) / ch) > 256) ch *= 2;
    return ch;
}
int64_t rank_chunks(int64_t B, int64_t N) {
    const int64_t ch = rank_chunk(B, N);
    return N > 0 ? (N + ch - 1) / ch : 1;
}

// A pass's key of entry i: the label itself, labels outside [0, V) as V (they
// sort last, as one more value).
__device__ __forceinline__ int32_t sort_key(int32_t l, int32_t V) { return (uint32_t)l < (uint32_t)V ? l : V; }

// The digit of a key: bits from `shift` on, `mask` of them (all, where one pass
// keeps a bin for each of the V + 1 keys).
__device__ __forceinline__ int32_t digit_of(int32_t k, int shift, int32_t mask) { return (k >> shift) & mask; }

// H[b][c][j]: entries of chunk c whose digit is j.  ROUTE: the digit is the
// label and labels outside [0, V) count nowhere.
template <bool ROUTE>
__global__ __launch_bounds__(kRankThreads) void k_digit_hist(const int32_t* __restrict__ keys, int64_t N, int32_t V,
                                                             int shift, int32_t mask, int K, int64_t CH, int64_t nch,
                                                             int32_t* __restrict__ H) {
    extern __shared__ int32_t s_h[];
    const int64_t b = blockIdx.y, c = blockIdx.x;
    const int64_t i0 = c * CH, i1 = i0 + CH < N ? i0 + CH : N;
    for (int j = threadIdx.x; j < K; j += kRankThreads) s_h[j] = 0;
    __syncthreads();
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kRankThreads) {
        const int32_t k = sort_key(keys[b * N + i], V);
        if (ROUTE) {
            if (k < V) atomicAdd(&s_h[k], 1);
        } else {
            atomicAdd(&s_h[digit_of(k, shift, mask)], 1);
        }
    }
    __syncthreads();
    int32_t* row = H + (b * nch + c) * (int64_t)K;
    for (int j = threadIdx.x; j < K; j += kRankThreads) row[j] = s_h[j];
}

// Places the entries of chunk c from base[j] = (bins before j) + P[c][j] on,
// in index order: wave w takes the w-th consecutive part of the chunk with a
// cursor table of its own in LDS, and the lanes of a round that hold the same
// digit find each other with one ballot per bit (lanes_matching_n).
// ROUTE: slots[i] = place (-1 for a label outside [0, V)), order[place] = i,
// and the block of chunk 0 stores offsets[0..K].
// Otherwise: keys_out[place] = key, idx_out[place] = idx_in[i] (idx_in NULL:
// i itself).
template <int NB, bool ROUTE>
__global__ __launch_bounds__(kRankThreads) void k_digit_rank(const int32_t* __restrict__ keys,
                                                             const int32_t* __restrict__ idx_in, int64_t N, int32_t V,
                                                             int shift, int32_t mask, int K, int64_t CH, int64_t nch,
                                                             const int32_t* __restrict__ P,
                                                             const int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ offsets,
                                                             int32_t* __restrict__ keys_out,
                                                             int32_t* __restrict__ idx_out,
                                                             int32_t* __restrict__ slots) {
    extern __shared__ int32_t s_tab[];  // [kRankWaves][K]
    __shared__ int32_t s_wave[3][kRankWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t b = blockIdx.y, c = blockIdx.x;
    const int64_t i0 = c * CH, i1 = i0 + CH < N ? i0 + CH : N;
    const int64_t part = ((i1 - i0 + kRankWaves - 1) / kRankWaves + 63) / 64 * 64;
    const int64_t w0 = i0 + w * part, w1 = w0 + part < i1 ? w0 + part : i1;
    int32_t* tab = s_tab + w * K;
    auto digit_at = [&](int64_t i, int32_t* key) {
        if (i >= w1) return -1;
        const int32_t k = sort_key(keys[b * N + i], V);
        *key = k;
        if (ROUTE) return k < V ? k : -1;
        return digit_of(k, shift, mask);
    };
    // the rows of counts and prefixes, kScanBins at a time, and the labels of a
    // short part are requested before anything waits
    constexpr int kScanBins = 3, kKeep = 2;
    int32_t cv[kScanBins], pv[kScanBins];
    auto get_bins = [&](int j0) {
#pragma unroll
        for (int e = 0; e < kScanBins; ++e) {
            const int j = j0 + e * kRankThreads + tid;
            cv[e] = j < K ? counts[b * K + j] : 0;
            pv[e] = j < K ? P[(b * nch + c) * (int64_t)K + j] : 0;
        }
    };
    get_bins(0);
    const bool keep = part <= 64 * kKeep;  // (block-uniform)
    int32_t kept_key[kKeep], kept_dg[kKeep];
    if (keep) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) kept_dg[u] = digit_at(w0 + u * 64 + lane, &kept_key[u]);
    }
    for (int j = lane; j < K; j += 64) tab[j] = 0;
    __builtin_amdgcn_wave_barrier();
    if (keep) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
            if (kept_dg[u] >= 0) atomicAdd(&tab[kept_dg[u]], 1);
    } else {
        for (int64_t r0 = w0; r0 < w1; r0 += 64) {
            int32_t key;
            const int32_t dg = digit_at(r0 + lane, &key);
            if (dg >= 0) atomicAdd(&tab[dg], 1);
        }
    }
    __syncthreads();
    int32_t carry = 0;
    for (int j0 = 0; j0 < K; j0 += kRankThreads * kScanBins) {  // (block-uniform)
        if (j0) get_bins(j0);
        int32_t incl[kScanBins];
#pragma unroll
        for (int e = 0; e < kScanBins; ++e) incl[e] = cv[e];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
#pragma unroll
            for (int e = 0; e < kScanBins; ++e) {
                const int32_t u = __shfl_up(incl[e], o, 64);
                if (lane >= o) incl[e] += u;
            }
        }
        if (lane == 63) {
#pragma unroll
            for (int e = 0; e < kScanBins; ++e) s_wave[e][w] = incl[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kScanBins; ++e) {
            const int j = j0 + e * kRankThreads + tid;
            int32_t before = carry + incl[e] - cv[e];
#pragma unroll
            for (int q = 0; q < kRankWaves; ++q) {
                before += q < w ? s_wave[e][q] : 0;
                carry += s_wave[e][q];
            }
            if (j < K) {
                if (ROUTE && c == 0) offsets[b * (K + 1) + j] = before;
                int32_t base = before + pv[e];
#pragma unroll
                for (int q = 0; q < kRankWaves; ++q) {
                    const int32_t n = s_tab[q * K + j];
                    s_tab[q * K + j] = base;
                    base += n;
                }
            }
        }
        __syncthreads();  // s_wave is rewritten, and the tables are read below
    }
    if (ROUTE && c == 0 && tid == 0) offsets[b * (K + 1) + K] = carry;
    auto place = [&](int64_t i, int32_t key, int32_t dg) {
        const bool ok = dg >= 0;
        const uint64_t m = lanes_matching_n<NB>(ok ? dg : 0, ok);
        const int rank = lanes_below(m);
        int32_t pos = -1;
        if (ok) {
            const int32_t at = tab[dg];
            pos = at + rank;
            if (rank == 0) tab[dg] = at + (int32_t)__popcll(m);
        }
        __builtin_amdgcn_wave_barrier();
        if (ROUTE) {
            if (i < w1) slots[b * N + i] = pos;
            if (ok) idx_out[b * N + pos] = (int32_t)i;
        } else if (ok) {
            keys_out[b * N + pos] = key;
            idx_out[b * N + pos] = idx_in ? idx_in[b * N + i] : (int32_t)i;
        }
    };
    if (keep) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) place(w0 + u * 64 + lane, kept_key[u], kept_dg[u]);
    } else {
        for (int64_t r0 = w0; r0 < w1; r0 += 64) {  // (wave-uniform)
            int32_t key = 0;
            const int32_t dg = digit_at(r0 + lane, &key);
            place(r0 + lane, key, dg);
        }
    }
}

template <bool ROUTE>
static hipError_t digit_pass(const int32_t* keys, const int32_t* idx_in, int64_t B, int64_t N, int32_t V, int shift,
                             int32_t mask, int K, int32_t* H, int32_t* P, int32_t* counts, int32_t* offsets, int32_t* keys_out,
                             int32_t* idx_out, int32_t* slots, hipStream_t s) {
    hipError_t e;
    const int64_t CH = rank_chunk(B, N), nch = rank_chunks(B, N);
    const dim3 grid((unsigned)nch, (unsigned)B);
    hipLaunchKernelGGL((k_digit_hist<ROUTE>), grid, dim3(kRankThreads), K * sizeof(int32_t), s, keys, N, V, shift, mask,
                       K, CH, nch, H);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_colscan(H, B, nch, K, P, counts, s)) != hipSuccess) return e;
    const size_t lds = (size_t)kRankWaves * K * sizeof(int32_t);
#define KM_GO(NB)                                                                                                  \
    do {                                                                                                           \
        if (lds > 64 * 1024 &&                                                                                     \
            (e = hipFuncSetAttribute((const void*)k_digit_rank<NB, ROUTE>, hipFuncAttributeMaxDynamicSharedMemorySize, \
                                     (int)lds)) != hipSuccess)                                                     \
            return e;                                                                                              \
        hipLaunchKernelGGL((k_digit_rank<NB, ROUTE>), grid, dim3(kRankThreads), lds, s, keys, idx_in, N, V, shift, \
                           mask, K, CH, nch, P, counts, offsets, keys_out, idx_out, slots);                              \
    } while (0)
    if (K <= 64) KM_GO(6);
    else if (K <= 512) KM_GO(9);
    else if (K <= 2048) KM_GO(11);
    else KM_GO(13);  // one pass over 4097 keys
#undef KM_GO
    return hipGetLastError();
}

hipError_t launch_route(const int32_t* experts, int64_t M, int64_t E, int32_t* H, int32_t* P, int32_t* counts,
                        int32_t* offsets, int32_t* slots, int32_t* order, hipStream_t s) {
    return digit_pass<true>(experts, nullptr, 1, M, (int32_t)E, 0, -1, (int)E, H, P, counts, offsets, nullptr, order, slots,
                            s);
}

// For every entry the count of the ones that sort before it: lower keys, and
// equal keys of lower index.  A block ranks 64 entries (a lane each); its 16
// waves split the problem's keys, read as LDS broadcasts.  In whole groups of
// 64 keys before or after the block's own the index order is known, so a
// key costs one compare and one add.
//
// The blocks after the ranking ones clear `clear_bytes` bytes a problem at
// `clear`, 64 KB each: memory the next launch wants zero, cleared beside the
// ranking instead of after it.
constexpr int kCountThreads = 1024;
constexpr int64_t kClearBlock = 65536;

__global__ __launch_bounds__(kCountThreads) void k_count_rank(const int32_t* __restrict__ labels, int64_t N,
                                                              int32_t V, int32_t* __restrict__ keys_out,
                                                              int32_t* __restrict__ idx_out, char* __restrict__ clear,
                                                              int64_t clear_bytes) {
    extern __shared__ __attribute__((aligned(16))) int32_t s_key[];  // [N rounded up to 64]
    __shared__ int32_t s_cnt[64];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int n = (int)N, n64 = (n + 63) / 64;
    const int64_t b = blockIdx.y;
    if ((int)blockIdx.x >= n64) {
        typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
        typedef i32x4 i32x4_any __attribute__((aligned(2)));
        typedef uint16_t u16_any;
        const int64_t c0 = (int64_t)(blockIdx.x - n64) * kClearBlock;
        char* p = clear + b * clear_bytes + c0;
        const int64_t m = clear_bytes - c0 < kClearBlock ? clear_bytes - c0 : kClearBlock;
        for (int64_t i = tid * 16; i + 16 <= m; i += kCountThreads * 16) *(i32x4_any*)(p + i) = i32x4{0, 0, 0, 0};
        if (tid < (m & 15) / 2) *(u16_any*)(p + (m & ~(int64_t)15) + tid * 2) = 0;  // (elements of two bytes or four)
        return;
    }
    for (int i = tid; i < n64 * 64; i += kCountThreads)
        s_key[i] = i < n ? sort_key(labels[b * N + i], V) : 0x7fffffff;
    if (tid < 64) s_cnt[tid] = 0;
    __syncthreads();
    const int me = blockIdx.x, i = me * 64 + lane;
    const int32_t key = s_key[i];
    int32_t cnt = 0;
    for (int g = w; g < n64; g += kCountThreads / 64) {  // groups of 64 keys (wave-uniform)
        const int4* k4 = (const int4*)(s_key + g * 64);
        if (g == me) {
            for (int j = 0; j < 64; ++j) {
                const int32_t o = s_key[g * 64 + j];
                cnt += o < key || (o == key && j < lane);
            }
        } else {
            const int32_t below = g < me ? key + 1 : key;  // key <= V < 2^31 - 1
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int4 o = k4[j];
                cnt += o.x < below;
                cnt += o.y < below;
                cnt += o.z < below;
                cnt += o.w < below;
            }
        }
    }
    atomicAdd(&s_cnt[lane], cnt);
    __syncthreads();
    if (w == 0 && i < n) {
        keys_out[b * N + s_cnt[lane]] = key;
        idx_out[b * N + s_cnt[lane]] = i;
    }
}

// The digits of a vocabulary's sort (labels plus the value V of the ones
// outside): one pass with a bin per key, or passes of equally many bits.
struct KeyDigits {
    int passes, bits, bins;
};
static KeyDigits key_digits(int64_t V) {
    if (V <= kRouteMaxE) return {1, 0, (int)V + 1};
    const int n = label_bits(V + 1), passes = (n + 11) / 12, bits = (n + passes - 1) / passes;
    return {passes, bits, 1 << bits};
}

// N^2 compares in one launch against three launches a pass.  A gradient by
// either, us a call: V = 1000 (one pass) N = 4096 18.2 and 20.1, N = 8192 23.7
// and 20.7; V = 32768 (two passes) N = 8192 30.9 and 37.4, N = 16384 47.4 and
// 41.6; V = 131072 N = 8192 29.9 and 50.2, N = 16384 54.6 and 52.2.
bool count_rank_fits(int64_t B, int64_t N, int64_t V) {
    return N <= (key_digits(V).passes > 1 ? 8192 : 4096) && B * N * N <= ((int64_t)1 << 27);
}

KeySortPlan plan_key_sort(int64_t B, int64_t N, int64_t V) {
    KeySortPlan p;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t BN = (size_t)B * N * sizeof(int32_t);
    p.keys = take(BN);
    p.order = take(BN);
    if (!count_rank_fits(B, N, V)) {
        const KeyDigits g = key_digits(V);
        const size_t rows = (size_t)B * rank_chunks(B, N) * g.bins * sizeof(int32_t);
        p.hist = take(rows);
        p.prefix = take(rows);
        p.counts = take((size_t)B * g.bins * sizeof(int32_t));
        if (g.passes > 1) {
            p.keys2 = take(BN);
            p.order2 = take(BN);
        }
    }
    p.total = off;
    return p;
}

hipError_t launch_key_sort(const int32_t* labels, int64_t B, int64_t N, int64_t V, const KeySortPlan& p, char* ws,
                           hipStream_t s, void* clear, int64_t clear_bytes) {
    if (B == 0 || N == 0) return hipSuccess;
    int32_t *keys = (int32_t*)(ws + p.keys), *order = (int32_t*)(ws + p.order);
    if (count_rank_fits(B, N, V)) {
        const int n64 = (int)((N + 63) / 64);
        const int64_t blocks = n64 + (clear ? (clear_bytes + kClearBlock - 1) / kClearBlock : 0);
        hipLaunchKernelGGL(k_count_rank, dim3((unsigned)blocks, (unsigned)B), dim3(kCountThreads),
                           (size_t)n64 * 64 * sizeof(int32_t), s, labels, N, (int32_t)V, keys, order, (char*)clear,
                           clear_bytes);
        return hipGetLastError();
    }
    const KeyDigits g = key_digits(V);
    int32_t *keys2 = (int32_t*)(ws + p.keys2), *order2 = (int32_t*)(ws + p.order2);
    const int32_t *kin = labels, *iin = nullptr;
    for (int q = 0; q < g.passes; ++q) {
        // the last pass lands in keys / order
        int32_t* ko = (g.passes - 1 - q) % 2 ? keys2 : keys;
        int32_t* io = (g.passes - 1 - q) % 2 ? order2 : order;
        const hipError_t e =
            digit_pass<false>(kin, iin, B, N, (int32_t)V, q * g.bits, g.passes > 1 ? g.bins - 1 : -1, g.bins, (int32_t*)(ws + p.hist),
                              (int32_t*)(ws + p.prefix), (int32_t*)(ws + p.counts), nullptr, ko, io, nullptr, s);
        if (e != hipSuccess) return e;
        kin = ko;
        iin = io;
    }
    return hipSuccess;
}

}  // namespace km

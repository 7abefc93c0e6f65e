// Gradient of the table of a lookup: per label, the scaled sum of the rows of
// the output's gradient that carry it; a label without a row gets zeros.
//
// The sort-inverse idea of the centroid update (technologypulse.uk
// "Flash-KMeans" article, bottleneck 2) for a table of any height and rows of
// any width: the labels are sorted (label_rank.hip), and the sorted rows are
// cut into pieces of TW.  A group of lanes walks one piece of one column
// slice, summing in float32 registers; a label that begins and ends in the
// piece is rounded and stored at once, so nothing but the gradient itself is
// written for it.  Sums of labels that cross a piece's border go to the
// piece's two float32 slots and are added in a fixed order by a second launch.
// No float atomics: the result is a function of the inputs alone.
//
// HBM bound: every row read once, every table row written once.  Rows of
// labels that do not occur are cleared by further blocks of the first launch,
// which find them by searching the sorted labels, so that no table of offsets
// is needed and the clearing runs beside the sums.  131072 rows of 4 KB into
// 131072: 220 us for 1069 MB, 4.9 TB/s, the rate of a copy.
#include "rows.h"

namespace km {

constexpr int kGradThreads = 256;

// First position of the sorted keys[0..n) whose key is at least v: a 64-way
// search by the whole wave.
__device__ __forceinline__ int64_t wave_lower_bound(const int32_t* __restrict__ keys, int64_t n, int64_t v,
                                                    int lane) {
    int64_t lo = 0, hi = n;  // keys before lo are < v, keys from hi on are >= v
    while (hi - lo > 64) {
        const int64_t step = (hi - lo) / 64;
        const int64_t at = lo + (lane + 1) * step - 1;
        const int c = (int)__popcll(__ballot(keys[at] < v));
        if (c < 64) hi = lo + (c + 1) * step - 1;
        lo += c * step;
    }
    return lo + (int64_t)__popcll(__ballot(lo + lane < hi && keys[lo + lane] < v));
}

// The group's piece: TW sorted rows from p * TW on, columns of chunk
// slice * GL + (lane in group).  slot[b][p][0]: the part of a label that began
// in an earlier piece; slot[b][p][1]: the part of one that goes on in the next.
template <typename TI, typename TO, int GL, bool STREAM>
__device__ __forceinline__ void reduce_piece(const TI* __restrict__ g, int64_t N, int d, int C,
                                             const int32_t* __restrict__ keys, const int32_t* __restrict__ order,
                                             int32_t V, int TW, int64_t p, int slice, int gl, float scale,
                                             TO* __restrict__ out, float* __restrict__ slot) {
    constexpr int VN = RowVec<TI>::N, U = 8;
    const int c = slice * GL + gl;
    const int64_t q0 = p * TW, q1 = q0 + TW < N ? q0 + TW : N;
    if (c >= C || q0 >= N) return;
    const int e0 = chunk_at<TI>(c, d);
    float acc[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) acc[i] = 0.f;
    int32_t cur = keys[q0];
    bool opens = q0 > 0 && keys[q0 - 1] == cur;
    auto store_slot = [&](int which) {
        float* to = slot + (p * 2 + which) * (int64_t)d + e0;
        store_f32<float, VN>(to, d, acc);
    };
    auto store_out = [&]() {
        float a[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) a[i] = scale * acc[i];
        store_f32<TO, VN, STREAM>(out + (int64_t)cur * d + e0, d, a);
    };
    for (int64_t q = q0; q < q1; q += U) {
        int32_t key[U], idx[U];
        typename RowVec<TI>::V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            key[u] = q + u < q1 ? keys[q + u] : V;
            idx[u] = q + u < q1 ? order[q + u] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = typename RowVec<TI>::V{};
            if (key[u] < V) v[u] = load_raw<TI>(g + (int64_t)idx[u] * d + e0, d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (q + u >= q1) continue;
            if (key[u] != cur) {
                // cur ended before this row
                if (cur < V) {
                    if (opens) store_slot(0);
                    else store_out();
                }
                opens = false;
                cur = key[u];
#pragma unroll
                for (int i = 0; i < VN; ++i) acc[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VN; ++i) acc[i] += elem_f32(v[u][i]);
        }
        if (cur >= V) return;  // keys are sorted: only rows without a label follow
    }
    if (opens) store_slot(0);
    else if (q1 < N && keys[q1] == cur) store_slot(1);
    else store_out();
}

// Clears the table rows [v0, v0 + RZ) that no label names.
template <typename TO, bool STREAM>
__device__ __forceinline__ void clear_rows(const int32_t* __restrict__ keys, int64_t N, int64_t V, int d, int64_t v0,
                                           int RZ, int lane, TO* __restrict__ out) {
    if (v0 >= V) return;
    const int nr = V - v0 < RZ ? (int)(V - v0) : RZ;
    const int64_t a = wave_lower_bound(keys, N, v0, lane), z = wave_lower_bound(keys, N, v0 + nr, lane);
    uint64_t empty = nr < 64 ? ((uint64_t)1 << nr) - 1 : ~(uint64_t)0;
    if (z > a) {
        // lane r looks for v0 + r among keys[a..z)
        int64_t lo = a, hi = z;
        const int64_t v = v0 + lane;
        while (lo < hi) {
            const int64_t m = (lo + hi) >> 1;
            if (keys[m] < v) lo = m + 1;
            else hi = m;
        }
        const bool there = lo < z && keys[lo] == v;
        empty &= ~(uint64_t)__ballot(there);
    }
    constexpr int VN = RowVec<TO>::N;
    while (empty) {  // runs of empty rows are contiguous in memory
        const int r = __builtin_ctzll(empty);
        const uint64_t rest = ~(empty >> r);
        const int len = rest ? __builtin_ctzll(rest) : 64 - r;
        TO* to = out + (v0 + r) * d;
        const int64_t n = (int64_t)len * d, nv = n / VN;
        for (int64_t i = lane; i < nv; i += 64)
            store_raw<TO, STREAM>(to + i * VN, VN, typename RowVec<TO>::V{});
        if (lane < n - nv * VN) to[nv * VN + lane] = TO{};
        empty &= len + r < 64 ? ~(uint64_t)0 << (len + r) : 0;
    }
}

template <typename TI, typename TO, int GL, bool STREAM>
__global__ __launch_bounds__(kGradThreads) void k_lookup_grad(const TI* __restrict__ g, int64_t N, int d, int C,
                                                              const int32_t* __restrict__ keys,
                                                              const int32_t* __restrict__ order, int64_t V, int TW,
                                                              int64_t npieces, int slices, int64_t red_blocks, int RZ,
                                                              float scale, TO* __restrict__ out,
                                                              float* __restrict__ slot) {
    const int64_t b = blockIdx.y;
    keys += b * N;
    out += b * V * d;
    if ((int64_t)blockIdx.x < red_blocks) {
        const int64_t gid = ((int64_t)blockIdx.x * kGradThreads + threadIdx.x) / GL;
        const int64_t p = gid / slices;
        if (p >= npieces) return;
        reduce_piece<TI, TO, GL, STREAM>(g + b * N * d, N, d, C, keys, order + b * N, (int32_t)V, TW, p,
                                 (int)(gid - p * slices), threadIdx.x % GL, scale, out,
                                 slot + b * npieces * 2 * (int64_t)d);
        return;
    }
    const int64_t wv = ((int64_t)blockIdx.x - red_blocks) * (kGradThreads / 64) + (threadIdx.x >> 6);
    clear_rows<TO, STREAM>(keys, N, V, d, wv * RZ, RZ, threadIdx.x & 63, out);
}

// Labels that cross piece borders.  A label that begins in piece p and reaches
// pieces p + 1 .. last has the row slot[p][1] + slot[p + 1][0] + .. +
// slot[last][0].  Up to kFoldShort pieces are added in that order by a group
// of GL lanes, one per (piece, column slice).  Longer runs are left to the
// blocks behind those, one per (kFoldShort pieces, column slice): at most one
// such run begins in them, the one that goes on past their end.  Its pieces are
// split over the block's waves, added in order within a wave and over
// the waves.
constexpr int kFoldShort = 16, kFoldU = 8;
// Wide rows have few slices a block could serve beside each other: big blocks.
constexpr int fold_threads(int GL) { return GL == 64 ? 1024 : 256; }

template <int VN>
__device__ __forceinline__ void add_slot(float (&acc)[VN], const float* __restrict__ from, int d) {
    if (d >= VN) {
#pragma unroll
        for (int i = 0; i < VN; ++i) acc[i] += from[i];
    } else {
        for (int i = 0; i < d; ++i) acc[i] += from[i];
    }
}

// slot[q][0] of the pieces q in [a, z), kFoldU of them in flight.
template <int VN>
__device__ __forceinline__ void add_slots(float (&acc)[VN], const float* __restrict__ slot, int64_t a, int64_t z,
                                          int e0, int d) {
    int64_t q = a;
    if (d >= VN) {
        for (; q + kFoldU <= z; q += kFoldU) {
            float v[kFoldU][VN];
#pragma unroll
            for (int u = 0; u < kFoldU; ++u)
#pragma unroll
                for (int i = 0; i < VN; ++i) v[u][i] = slot[(q + u) * 2 * (int64_t)d + e0 + i];
#pragma unroll
            for (int u = 0; u < kFoldU; ++u)
#pragma unroll
                for (int i = 0; i < VN; ++i) acc[i] += v[u][i];
        }
    }
    for (; q < z; ++q) add_slot<VN>(acc, slot + q * 2 * (int64_t)d + e0, d);
}

template <typename TI, typename TO, int GL>
__global__ __launch_bounds__(fold_threads(GL)) void k_lookup_grad_fold(const int32_t* __restrict__ keys, int64_t N, int d,
                                                                   int C, int64_t V, int TW, int64_t npieces,
                                                                   int slices, int64_t short_blocks, int long_slices,
                                                                   float scale, TO* __restrict__ out,
                                                                   const float* __restrict__ slot) {
    constexpr int VN = RowVec<TI>::N, FT = fold_threads(GL), NW = FT / 64;
    __shared__ float s_acc[NW][64][VN + 1];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t b = blockIdx.y;
    keys += b * N;
    slot += b * npieces * 2 * (int64_t)d;
    out += b * V * d;
    float acc[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) acc[i] = 0.f;
    if ((int64_t)blockIdx.x < short_blocks) {
        const int64_t gid = ((int64_t)blockIdx.x * FT + threadIdx.x) / GL, p = gid / slices;
        const int c = (int)(gid - p * slices) * GL + threadIdx.x % GL;
        if (p + 1 >= npieces || c >= C) return;
        const int64_t q0 = p * TW, q1 = q0 + TW;
        const int32_t v = keys[q1 - 1];
        if (v >= V || keys[q1] != v || (q0 > 0 && keys[q0 - 1] == v)) return;  // nothing begins here and goes on
        // how many of the next kFoldShort + 1 pieces begin with v (the first ones, as keys are sorted)
        int n = 0;
#pragma unroll
        for (int i = 1; i <= kFoldShort + 1; ++i) {
            const int64_t q = p + i < npieces ? p + i : npieces - 1;
            n += p + i < npieces && keys[q * TW] == v;
        }
        if (n > kFoldShort) return;
        const int e0 = chunk_at<TI>(c, d);
        add_slot<VN>(acc, slot + (p * 2 + 1) * (int64_t)d + e0, d);
        add_slots<VN>(acc, slot, p + 1, p + 1 + n, e0, d);
#pragma unroll
        for (int i = 0; i < VN; ++i) acc[i] *= scale;
        store_f32<TO, VN>(out + (int64_t)v * d + e0, d, acc);
        return;
    }
    const int64_t id = (int64_t)blockIdx.x - short_blocks, grp = id / long_slices;
    const int c = (int)(id - grp * long_slices) * 64 + lane;
    const int64_t pe = (grp + 1) * kFoldShort;  // the first piece after the block's
    if (pe >= npieces) return;
    const int32_t v = keys[pe * TW];
    if (v >= V || keys[pe * TW - 1] != v) return;
    // lane i: does v come from before piece pe - 1 - i?  The first lane that says no is the piece it begins in
    const int64_t back = pe - 1 - lane;
    const uint64_t here = __ballot(lane < kFoldShort && (back == 0 || keys[back * TW - 1] != v));
    if (!here) return;  // it begins before the block's pieces
    const int64_t p = pe - 1 - __builtin_ctzll(here);
    const int64_t q1 = pe * TW, end = q1 + wave_lower_bound(keys + q1, N - q1, (int64_t)v + 1, lane);
    const int64_t last = (end - 1) / TW;
    if (last - p <= kFoldShort) return;
    const bool live = c < C;
    const int e0 = live ? chunk_at<TI>(c, d) : 0;
    const int64_t per = (last - p + NW - 1) / NW, a = p + 1 + w * per, z = a + per < last + 1 ? a + per : last + 1;
    if (live) {
        if (w == 0) add_slot<VN>(acc, slot + (p * 2 + 1) * (int64_t)d + e0, d);
        add_slots<VN>(acc, slot, a, z, e0, d);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) s_acc[w][lane][i] = acc[i];
    __syncthreads();
    if (w == 0 && live) {
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            float t = acc[i];
#pragma unroll
            for (int q = 1; q < NW; ++q) t += s_acc[q][lane][i];
            acc[i] = scale * t;
        }
        store_f32<TO, VN>(out + (int64_t)v * d + e0, d, acc);
    }
}

// Sorted rows per piece: long pieces write fewer slots, short ones make more
// waves.  8 rows (one batch of loads) and doubled, to 256 at most, while 4096
// waves remain (2048 waves: 257 us against 222 for 131072 rows of 4 KB, and
// 15.8 against 12.7 for 8 x 16411 rows of 260 bytes; at least 16 rows: 11.0
// against 6.8 for 2000 rows of 2 KB).
static int grad_tw(int64_t B, int64_t N, int64_t slices_waves64) {
    int tw = 8;
    while (tw < 256 && B * (N / (2 * tw)) * slices_waves64 >= 4096 * 64) tw *= 2;
    return tw;
}

static int group_lanes(int C) { return C <= 8 ? 8 : C <= 16 ? 16 : C <= 32 ? 32 : 64; }

LookupGradPlan plan_lookup_grad(int64_t B, int64_t N, int64_t d, int64_t V, DType xt) {
    LookupGradPlan p;
    const int C = row_chunks(d, dtype_bytes(xt)), GL = group_lanes(C);
    p.tw = grad_tw(B, N, (int64_t)((C + GL - 1) / GL) * GL);
    p.npieces = N > 0 ? (N + p.tw - 1) / p.tw : 0;
    p.sort = plan_key_sort(B, N, V);
    p.slot = p.sort.total;
    p.total = p.slot + (p.npieces > 1 ? (((size_t)B * p.npieces * 2 * d * sizeof(float) + 255) & ~(size_t)255) : 0);
    return p;
}

template <typename TI, typename TO>
static hipError_t grad_launch(const TI* g, int64_t B, int64_t N, int64_t d, const int32_t* keys, const int32_t* order,
                              int64_t V, const LookupGradPlan& p, float scale, TO* out, float* slot, bool cleared,
                              hipStream_t s) {
    const int C = row_chunks(d, sizeof(TI)), GL = group_lanes(C);
    const int slices = (C + GL - 1) / GL;
    const int64_t red = (p.npieces * slices * GL + kGradThreads - 1) / kGradThreads;
    // a clearing wave takes up to 64 KB of rows
    int64_t rz = 65536 / (d * (int64_t)sizeof(TO));
    rz = rz < 1 ? 1 : rz > 64 ? 64 : rz;
    const int64_t clr = cleared ? 0 : ((V + rz - 1) / rz + kGradThreads / 64 - 1) / (kGradThreads / 64);
    const dim3 grid((unsigned)(red + clr), (unsigned)B);
    const bool stream = stream_out(B * V * d * (int64_t)sizeof(TO));
#define KM_GO2(G, ST)                                                                                                 \
    hipLaunchKernelGGL((k_lookup_grad<TI, TO, G, ST>), grid, dim3(kGradThreads), 0, s, g, N, (int)d, C, keys, order, V, \
                       p.tw, p.npieces, slices, red, (int)rz, scale, out, slot)
#define KM_GO(G)                     \
    do {                             \
        if (stream) KM_GO2(G, true); \
        else KM_GO2(G, false);       \
    } while (0)
    if (GL == 8) KM_GO(8);
    else if (GL == 16) KM_GO(16);
    else if (GL == 32) KM_GO(32);
    else KM_GO(64);
#undef KM_GO
#undef KM_GO2
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.npieces < 2) return e;
    const int ls = (C + 63) / 64;
    const int64_t ft = fold_threads(GL), sb = ((p.npieces - 1) * slices * GL + ft - 1) / ft;
    const int64_t lb = (p.npieces - 1) / kFoldShort * ls;
#define KM_GO(G)                                                                                                     \
    hipLaunchKernelGGL((k_lookup_grad_fold<TI, TO, G>), dim3((unsigned)(sb + lb), (unsigned)B), dim3((unsigned)ft),  \
                       0, s, keys, N, (int)d, C, V, p.tw, p.npieces, slices, sb, ls, scale, out, slot)
    if (GL == 8) KM_GO(8);
    else if (GL == 16) KM_GO(16);
    else if (GL == 32) KM_GO(32);
    else KM_GO(64);
#undef KM_GO
    return hipGetLastError();
}

hipError_t launch_lookup_grad(DType xt, const void* g, int64_t B, int64_t N, int64_t d, const int32_t* labels,
                              int64_t V, float scale, DType gt, void* out, const LookupGradPlan& p, char* ws,
                              hipStream_t s) {
    if (B == 0) return hipSuccess;
    // Few rows for the table's height: the whole gradient is cleared beside the
    // one launch that ranks the labels (up to a quarter of the table written
    // twice costs less than the search for the rows to clear), where one launch
    // has the threads for it (1024 for 64 KB).
    const int64_t bytes = V * d * dtype_bytes(gt);
    const bool cleared = N > 0 && count_rank_fits(B, N, V) && 4 * N <= V && bytes < (int64_t)1 << 37;
    const hipError_t e = launch_key_sort(labels, B, N, V, p.sort, ws, s, cleared ? out : nullptr, bytes);
    if (e != hipSuccess) return e;
    const int32_t *keys = (int32_t*)(ws + p.sort.keys), *order = (int32_t*)(ws + p.sort.order);
    float* slot = (float*)(ws + p.slot);
#define KM_GO(TI, TO) \
    return grad_launch<TI, TO>((const TI*)g, B, N, d, keys, order, V, p, scale, (TO*)out, slot, cleared, s)
    if (xt == DType::F32) KM_GO(float, float);
    if (xt == DType::F16) {
        if (gt == DType::F32) KM_GO(_Float16, float);
        KM_GO(_Float16, _Float16);
    }
    if (gt == DType::F32) KM_GO(uint16_t, float);
    KM_GO(uint16_t, uint16_t);
#undef KM_GO
}

}  // namespace km

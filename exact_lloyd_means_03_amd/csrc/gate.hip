// The gate of a layer of experts: the softmax of every token's logits, its
// largest ones in order, the choices counted, the loss that balances the
// experts, and the gradient of all of it.
//
// A row of E logits is held by a group of L lanes (16 up to 256 experts, so that
// every exchange is a DPP move inside 16 lanes; 64 beyond), expert j L + lane in
// register j.  Up to 16 choices of up to 256 experts are ranked at once (gate_pick);
// otherwise choosing is `top` rounds of two reductions: the largest key of the
// group, then the lowest expert that has it.
//
// Vector instructions bound both kernels: 16421 rows of 256 float32 logits, 8
// choices (17 MB, 3.5 us of memory): 13.9 us and 5.2 for the fold of the blocks'
// parts (in rounds: 17.8); their gradient 11 us.  24 rows of 64: 4 us, one launch.
#include "codes8.h"

namespace km {

constexpr int kGateTopMax = 64;
constexpr int gate_threads(int L) { return L == 16 ? 512 : 256; }  // blocks of 32 rows, or of 4
bool gate_top_fits(int64_t top) { return top <= kGateTopMax; }

// A logit as a number that orders like it: 0 for those that are never chosen
// (-infinity, NaN), equal for the two zeros.
__device__ __forceinline__ uint32_t gate_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.f);
    return l > -INFINITY ? ((int32_t)u < 0 ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float gate_value(uint32_t key) {
    return __uint_as_float((int32_t)key < 0 ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const _Float16* p) { return (float)*p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }

// exp(x) for x <= 0 (NaN stays): 2^(x log2 e) with the product's own rounding added
// back, 2 units in the last place in half the instructions of expf; 0 below 2^-126.
__device__ __forceinline__ float gate_exp(float x) {
    x = x < -150.f ? -150.f : x;
    const float t = x * 1.44269502f, rest = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -t));
    const float r = __builtin_amdgcn_exp2f(t);
    return fmaf(r, rest * 0.693147182f, r);
}

// z[j] = exp(l[j] - m), m the largest logit that is a number; returns 1 / sum z
// (0 for a row of -infinity; NaN where a logit is NaN or +infinity).
template <int L, int EPL>
__device__ __forceinline__ float gate_softmax(const float (&l)[EPL], float (&z)[EPL], float* m_out) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);  // (NaN is passed over)
    m = __uint_as_float(lane_fold<L>(__float_as_uint(m), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
    m = m > -INFINITY ? m : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        z[j] = gate_exp(l[j] - m);
        sum += z[j];
    }
    sum = lane_sum<L>(sum);
    *m_out = m;
    return sum == 0.f ? 0.f : 1.f / sum;
}

// The `top` <= 16 largest of a row's keys at once.  The top-th largest of the lanes'
// maxima bounds the choices from below; the few keys that reach it (a dozen of 256
// where top is 8) are gathered, one a lane, and each lane counts the ones that come
// before its own.  False where a row of the wave has more than 16 such keys (ties,
// rows with few lanes left).  s: the group's 16 places.
struct GatePick {
    uint32_t key, e;  // the lane's (0: none)
    int rank, total;  // its place, and the gathered ones
};
template <int N, typename F>
__device__ __forceinline__ void each_rotation(F f) {  // f of the number of lanes turned: 1 .. 15
    if constexpr (N < 16) {
        f(Int<N>{});
        each_rotation<N + 1>(f);
    }
}
template <int EPL>
__device__ __forceinline__ bool gate_pick(const uint32_t (&key)[EPL], int lane, int top, uint2* s, GatePick* p) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = best > key[j] ? best : key[j];
    int c = 1;  // maxima that are not below the lane's
    each_rotation<1>([&](auto n) { c += dpp<0x120 + decltype(n)::value>(best) >= best; });
    const uint32_t bound = lane_max<16>(c >= top ? best : 0u), least = bound ? bound : 1u;
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) n += key[j] >= least;
    uint32_t upto = n;  // with the lanes before
    upto += dpp<0x111>(upto);
    upto += dpp<0x112>(upto);
    upto += dpp<0x114>(upto);
    upto += dpp<0x118>(upto);
    p->total = (int)lane_max<16>(upto);
    if (__ballot(p->total > 16)) return false;
    uint32_t at = upto - n;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (key[j] >= least) s[at++] = uint2{key[j], (uint32_t)(j * 16 + lane)};
    __builtin_amdgcn_wave_barrier();
    const uint2 mine = s[lane];
    p->key = lane < p->total ? mine.x : 0u;
    p->e = mine.y;
    p->rank = 0;
    each_rotation<1>([&](auto n) {
        const uint32_t k = dpp<0x120 + decltype(n)::value>(p->key), e = dpp<0x120 + decltype(n)::value>(p->e);
        p->rank += (k > p->key) | ((k == p->key) & (e < p->e));
    });
    __builtin_amdgcn_wave_barrier();  // (read before the next row's are written)
    return true;
}

// E sum_e shares[e] counts[e] / sum(counts) from dot = sum_e shares[e] counts[e]
// (NaN shares make a NaN loss, also where no expert could be chosen).
__device__ __forceinline__ float gate_loss(float dot, int64_t choices, int E) {
    return choices ? dot * ((float)E / (float)choices) : dot * 0.f;
}

struct GateSum {
    float dot;
    int32_t all;
};

// Blocks of the gate leave their counts and probabilities' sums: part_n[b][E + 1]
// (the last one: rows that are not all -infinity) and part_p[b][E].  A single
// block has them all and finishes by itself.
template <typename T, int L, int EPL, int KR>
__global__ __launch_bounds__(gate_threads(L)) void k_gate(const T* __restrict__ logits, int64_t Tn, int E, int top,
                                                       bool normalize, int32_t* __restrict__ experts,
                                                       float* __restrict__ weights, int32_t* __restrict__ part_n,
                                                       float* __restrict__ part_p, int32_t* __restrict__ ticket,
                                                       int32_t* __restrict__ counts, float* __restrict__ shares,
                                                       float* __restrict__ loss) {
    constexpr int NT = gate_threads(L), G = NT / L, GW = 64 / L, W = NT / 64;
    constexpr bool PICK = L == 16 && KR == 1;
    __shared__ uint2 s_pick[PICK ? G : 1][16];
    extern __shared__ int32_t s_cnt[];  // [E + 1]; then float [W][E]
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    for (int j = tid; j <= E; j += NT) s_cnt[j] = 0;
    __syncthreads();
    float acc[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
    int rows = 0;
    // (whole waves run each round: a group behind the last row takes part without one)
    for (int64_t t0 = (int64_t)blockIdx.x * G; t0 < Tn; t0 += (int64_t)gridDim.x * G) {
        const int64_t t = t0 + grp;
        const bool in = t < Tn;
        float l[EPL], z[EPL], m;
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * L + lane;
            l[j] = in && e < E ? load_logit(logits + t * E + e) : -INFINITY;
            key[j] = gate_key(l[j]);
        }
        const float inv = gate_softmax<L, EPL>(l, z, &m);
        if (inv != 0.f) {
            rows += lane == 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] = fmaf(z[j], inv, acc[j]);
        }
        if constexpr (PICK) {
            GatePick p;
            if (gate_pick<EPL>(key, lane, top, s_pick[grp], &p)) {
                const bool chosen = p.key && p.rank < top;
                const float zk = chosen ? gate_exp(gate_value(p.key) - m) : 0.f;
                const float sum = lane_sum<16>(zk), by = !normalize ? inv : sum == 0.f ? 0.f : 1.f / sum;
                if (chosen) {
                    atomicAdd(&s_cnt[p.e], 1);
                    experts[t * top + p.rank] = (int32_t)p.e;
                    weights[t * top + p.rank] = zk * by;
                }
                if (in && lane >= p.total && lane < top) {
                    experts[t * top + lane] = -1;
                    weights[t * top + lane] = 0.f;
                }
                continue;
            }
        }
        uint32_t kk[KR], ke[KR];  // the choice k is lane k % L's: its key (0: none) and expert
#pragma unroll
        for (int u = 0; u < KR; ++u) kk[u] = 0, ke[u] = ~0u;
        for (int k = 0; k < top; ++k) {
            uint32_t most = 0, at = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) most = most > key[j] ? most : key[j];
            most = lane_max<L>(most);
#pragma unroll
            for (int j = EPL - 1; j >= 0; --j) at = key[j] == most ? (uint32_t)(j * L + lane) + 1 : at;
            const uint32_t e = lane_min<L>(at - 1);  // (a lane without it: the largest number)
            if (most && e % L == (uint32_t)lane) atomicAdd(&s_cnt[e], 1);
            uint32_t gone = most && e % L == (uint32_t)lane ? e / L : ~0u;
            asm("" : "+v"(gone));  // (one comparison for each register below)
#pragma unroll
            for (int j = 0; j < EPL; ++j) key[j] = gone == (uint32_t)j ? 0u : key[j];
#pragma unroll
            for (int u = 0; u < KR; ++u) {
                const bool here = k == u * L + lane;
                kk[u] = here ? most : kk[u];
                ke[u] = here && most ? e : ke[u];
            }
        }
        float zk[KR], sum = 0.f;
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            zk[u] = kk[u] ? gate_exp(gate_value(kk[u]) - m) : 0.f;
            sum += zk[u];
        }
        sum = lane_sum<L>(sum);
        const float by = !normalize ? inv : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            const int k = u * L + lane;
            if (in && k < top) {
                experts[t * top + k] = (int32_t)ke[u];
                weights[t * top + k] = kk[u] ? zk[u] * by : 0.f;
            }
        }
    }
    // the groups of a wave, then the waves, in order
    float* s_p = (float*)(s_cnt + E + 1);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        if constexpr (GW > 1) {
            acc[j] += __shfl_xor(acc[j], 16, 64);
            acc[j] += __shfl_xor(acc[j], 32, 64);
        }
        const int e = j * L + lane;
        if ((tid & 63) < L && e < E) s_p[(tid >> 6) * E + e] = acc[j];
    }
    if (rows) atomicAdd(&s_cnt[E], rows);
    __syncthreads();
    if (gridDim.x == 1) {
        const int32_t n = s_cnt[E];
        const float inv = n ? 1.f / (float)n : 0.f;
        float dot = 0.f;
        int32_t all = 0;
        for (int e = tid; e < E; e += NT) {
            float p = s_p[e];
            for (int i = 1; i < W; ++i) p += s_p[i * E + e];
            p *= inv;
            counts[e] = s_cnt[e];
            shares[e] = p;
            all += s_cnt[e];
            dot = fmaf((float)s_cnt[e], p, dot);
        }
        if (tid == 0) counts[E] = n;
        dot = lane_sum<64>(dot);
        all = (int32_t)lane_fold<64>((uint32_t)all, [](uint32_t a, uint32_t b) { return a + b; });
        __shared__ GateSum s_sum[W];
        if ((tid & 63) == 0) s_sum[tid >> 6] = {dot, all};
        __syncthreads();
        if (tid == 0) {
            int64_t c = 0;
            dot = 0.f;
            for (int i = 0; i < W; ++i) dot += s_sum[i].dot, c += s_sum[i].all;
            loss[0] = gate_loss(dot, c, E);
        }
        return;
    }
    if (blockIdx.x == 0 && tid == 0) *ticket = 0;
    int32_t* pn = part_n + (int64_t)blockIdx.x * (E + 1);
    float* pp = part_p + (int64_t)blockIdx.x * E;
    for (int e = tid; e <= E; e += NT) {
        pn[e] = s_cnt[e];
        if (e < E) {
            float p = s_p[e];
            for (int i = 1; i < W; ++i) p += s_p[i * E + e];
            pp[e] = p;
        }
    }
}

// Counts and shares of the blocks' parts, 16 experts a block: 64 groups of 16
// threads take every 64th part, then their sums in order.  The block that comes
// last adds all blocks' parts of the loss, in order.
constexpr int kFoldExperts = 16, kFoldParts = 64;

__global__ __launch_bounds__(kFoldExperts* kFoldParts) void k_gate_fold(
    const int32_t* __restrict__ part_n, const float* __restrict__ part_p, int nblk, int E, GateSum* __restrict__ sums,
    int32_t* __restrict__ ticket, int32_t* __restrict__ counts, float* __restrict__ shares, float* __restrict__ loss) {
    constexpr int W = kFoldExperts * kFoldParts / 64;
    __shared__ float s_p[W][kFoldExperts];
    __shared__ int32_t s_c[W][kFoldExperts], s_n[W];
    const int tid = threadIdx.x, j = tid % kFoldExperts, h = tid / kFoldExperts;
    const int e = blockIdx.x * kFoldExperts + j;
    float p = 0.f;
    int32_t c = 0, n = 0;
    const int at = e < E ? e : E - 1;
    constexpr int U = 8;  // parts in flight: their loads are what a block waits for
    for (int b0 = h; b0 < nblk; b0 += U * kFoldParts) {
        float pv[U];
        int32_t cv[U], nv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kFoldParts < nblk ? b0 + u * kFoldParts : b0;
            pv[u] = part_p[(int64_t)b * E + at];
            cv[u] = part_n[(int64_t)b * (E + 1) + at];
            nv[u] = part_n[(int64_t)b * (E + 1) + E];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u * kFoldParts < nblk) p += pv[u], c += cv[u], n += j == 0 ? nv[u] : 0;
        }
    }
    auto over = [&]() {  // the four parts of a wave
        p += __shfl_xor(p, 16, 64);
        c += __shfl_xor(c, 16, 64);
        n += __shfl_xor(n, 16, 64);
        p += __shfl_xor(p, 32, 64);
        c += __shfl_xor(c, 32, 64);
        n += __shfl_xor(n, 32, 64);
    };
    over();
    if ((tid & 63) < kFoldExperts) s_p[tid >> 6][j] = p, s_c[tid >> 6][j] = c;
    if ((tid & 63) == 0) s_n[tid >> 6] = n;
    __syncthreads();
    if (tid < 64) {  // the first wave: lane j an expert, four quarters of the waves
        p = 0.f;
        c = n = 0;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) p += s_p[h * (W / 4) + i][j], c += s_c[h * (W / 4) + i][j], n += s_n[h * (W / 4) + i];
        over();
        if (tid < kFoldExperts && e < E) {
            p *= n ? 1.f / (float)n : 0.f;
            counts[e] = c;
            shares[e] = p;
        } else {
            p = 0.f;
            c = 0;
        }
        const float dot = lane_sum<64>((float)c * p);
        c = (int32_t)lane_fold<64>((uint32_t)c, [](uint32_t a, uint32_t b) { return a + b; });
        int last = 0;
        if (tid == 0) {
            if (blockIdx.x == 0) counts[E] = n;
            __hip_atomic_store(&sums[blockIdx.x].dot, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&sums[blockIdx.x].all, c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        }
        if (__builtin_amdgcn_readfirstlane(last)) {
            float d = 0.f;
            int32_t a = 0;  // (choices: fewer than 2^31)
            for (int i = tid; i < (int)gridDim.x; i += 64) {
                d += __hip_atomic_load(&sums[i].dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                a += __hip_atomic_load(&sums[i].all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            d = lane_sum<64>(d);
            a = (int32_t)lane_fold<64>((uint32_t)a, [](uint32_t x, uint32_t y) { return x + y; });
            if (tid == 0) loss[0] = gate_loss(d, a, E);
        }
    }
}

static int64_t gate_rows(int64_t E) { return E <= 256 ? gate_threads(16) / 16 : gate_threads(64) / 64; }

// Blocks of the gate: one where few rows make at most two rounds of it (a second
// launch costs more), else one for every round of rows, as far as their parts are
// no more than 4 MB or 256 rows of them.
static int64_t gate_blocks(int64_t T, int64_t E) {
    const int64_t rows = gate_rows(E), n = (T + rows - 1) / rows;
    if (n <= 2) return 1;
    int64_t most = ((int64_t)1 << 19) / E;
    most = most < 256 ? 256 : most > 2048 ? 2048 : most;
    const int64_t rounds = (n + most - 1) / most;
    return (n + rounds - 1) / rounds;
}
struct GatePlan {
    size_t part_n = 0, part_p = 0, sums = 0, ticket = 0, total = 0;
};
static GatePlan plan_gate(int64_t T, int64_t E) {
    GatePlan p;
    const int64_t nblk = gate_blocks(T, E);
    if (nblk == 1) return p;
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    p.part_p = up((size_t)nblk * (E + 1) * sizeof(int32_t));
    p.sums = p.part_p + up((size_t)nblk * E * sizeof(float));
    p.ticket = p.sums + up((size_t)((E + kFoldExperts - 1) / kFoldExperts) * sizeof(GateSum));
    p.total = p.ticket + 256;
    return p;
}
size_t gate_scratch(int64_t T, int64_t E) { return plan_gate(T, E).total; }

#define KM_GATE(T)                          \
    do {                                    \
        if (E <= 16) KM_GO(T, 16, 1);       \
        else if (E <= 32) KM_GO(T, 16, 2);  \
        else if (E <= 64) KM_GO(T, 16, 4);  \
        else if (E <= 128) KM_GO(T, 16, 8); \
        else if (E <= 256) KM_GO(T, 16, 16); \
        else if (E <= 512) KM_GO(T, 64, 8); \
        else if (E <= 1024) KM_GO(T, 64, 16); \
        else if (E <= 2048) KM_GO(T, 64, 32); \
        else KM_GO(T, 64, 64);              \
    } while (0)

hipError_t launch_gate(DType xt, const void* logits, int64_t T, int64_t E, int64_t top, bool normalize, int32_t* experts,
                       float* weights, int32_t* counts, float* shares, float* loss, void* ws, hipStream_t s) {
    const int64_t nblk = gate_blocks(T, E);
    const GatePlan p = plan_gate(T, E);
    int32_t* pn = (int32_t*)((char*)ws + p.part_n);
    float* pp = (float*)((char*)ws + p.part_p);
    int32_t* ticket = (int32_t*)((char*)ws + p.ticket);
    const size_t lds = (size_t)(E + 1 + (E <= 256 ? gate_threads(16) : gate_threads(64)) / 64 * E) * sizeof(int32_t);
    hipError_t e = hipSuccess;
#define KM_GO2(TT, L, EPL, KR)                                                                                         \
    do {                                                                                                               \
        if (lds > 64 * 1024 && (e = hipFuncSetAttribute((const void*)k_gate<TT, L, EPL, KR>,                           \
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)) != hipSuccess) \
            return e;                                                                                                  \
        hipLaunchKernelGGL((k_gate<TT, L, EPL, KR>), dim3((unsigned)nblk), dim3(gate_threads(L)), lds, s,              \
                           (const TT*)logits, T, (int)E, (int)top, normalize, experts, weights, pn, pp, ticket,        \
                           counts, shares, loss);                                                                      \
    } while (0)
#define KM_GO(TT, L, EPL)                               \
    do {                                                \
        if (top <= L) KM_GO2(TT, L, EPL, 1);            \
        else KM_GO2(TT, L, EPL, kGateTopMax / L);       \
    } while (0)
    if (xt == DType::F32) KM_GATE(float);
    else if (xt == DType::F16) KM_GATE(_Float16);
    else KM_GATE(uint16_t);
#undef KM_GO
#undef KM_GO2
    if ((e = hipGetLastError()) != hipSuccess || nblk == 1) return e;
    hipLaunchKernelGGL(k_gate_fold, dim3((unsigned)((E + kFoldExperts - 1) / kFoldExperts)),
                       dim3(kFoldExperts * kFoldParts), 0, s, pn, pp, (int)nblk, (int)E, (GateSum*)((char*)ws + p.sums),
                       ticket, counts, shares, loss);
    return hipGetLastError();
}

// The gradient.  The chosen experts' part reaches the lane that owns the expert
// through LDS: a group writes its row, the lanes of the choices add to it, the
// group reads it back.
template <typename T, int L, int EPL>
__global__ __launch_bounds__(gate_threads(L)) void k_gate_grad(const T* __restrict__ logits, int64_t Tn, int E, int top,
                                                            bool normalize, const int32_t* __restrict__ experts,
                                                            const int32_t* __restrict__ counts,
                                                            const float* __restrict__ gweights,
                                                            const float* __restrict__ gloss, T* __restrict__ out) {
    constexpr int G = gate_threads(L) / L, KR = kGateTopMax / L;
    extern __shared__ float s_row[];  // [G][EPL L]
    const int lane = threadIdx.x & (L - 1), grp = threadIdx.x / L;
    float* row = s_row + grp * EPL * L;
    float f[EPL];
    {
        int32_t all = 0;
        float c[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * L + lane;
            const int32_t n = gloss && e < E ? counts[e] : 0;
            all += n;
            c[j] = (float)n;
        }
        all = (int32_t)lane_fold<L>((uint32_t)all, [](uint32_t a, uint32_t b) { return a + b; });
        const float by = gloss && all > 0 ? gloss[0] * (float)E / ((float)counts[E] * (float)all) : 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) f[j] = gloss && all > 0 ? by * c[j] : 0.f;
    }
    for (int64_t t0 = (int64_t)blockIdx.x * G; t0 < Tn; t0 += (int64_t)gridDim.x * G) {
        const int64_t t = t0 + grp;
        const bool in = t < Tn;
        float l[EPL], z[EPL], m;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * L + lane;
            l[j] = in && e < E ? load_logit(logits + t * E + e) : -INFINITY;
        }
        int32_t ek[KR];
        float gk[KR], lk[KR];
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            const int k = u * L + lane;
            const bool on = in && k < top && gweights;
            ek[u] = on ? experts[t * top + k] : -1;
            gk[u] = on ? gweights[t * top + k] : 0.f;
            if ((uint32_t)ek[u] >= (uint32_t)E) ek[u] = -1;
            lk[u] = ek[u] >= 0 ? load_logit(logits + t * E + ek[u]) : -INFINITY;
        }
        const float inv = gate_softmax<L, EPL>(l, z, &m);
        // the choices' softmax numerators, and <w, gw> over the chosen
        float wk[KR], sum = 0.f, dot = 0.f;
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            wk[u] = ek[u] >= 0 ? gate_exp(lk[u] - m) : 0.f;
            sum += wk[u];
            if (ek[u] >= 0) dot = fmaf(wk[u], gk[u], dot);
        }
        sum = lane_sum<L>(sum);
        dot = lane_sum<L>(dot);
        const float by = normalize ? (sum == 0.f ? 0.f : 1.f / sum) : inv;
        dot *= by;
        float pf = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) pf = fmaf(z[j] * inv, f[j], pf);
        pf = lane_sum<L>(pf);
        const float less = normalize ? pf : pf + dot;
#pragma unroll
        for (int j = 0; j < EPL; ++j) row[j * L + lane] = inv == 0.f ? 0.f : z[j] * inv * (f[j] - less);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < KR; ++u)
            if (ek[u] >= 0) atomicAdd(&row[ek[u]], wk[u] * by * (normalize ? gk[u] - dot : gk[u]));
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * L + lane;
            const float v = row[j * L + lane];
            if (in && e < E) out[t * E + e] = elem_from<T>(v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

hipError_t launch_gate_grad(DType xt, const void* logits, int64_t T, int64_t E, int64_t top, bool normalize,
                            const int32_t* experts, const int32_t* counts, const float* gweights, const float* gloss,
                            void* out, hipStream_t s) {
    if (T == 0) return hipSuccess;
    const int64_t rows = gate_rows(E), n = (T + rows - 1) / rows;
    const unsigned nblk = (unsigned)(n < 2048 ? n : 2048);
    hipError_t e = hipSuccess;
#define KM_GO(TT, L, EPL)                                                                                              \
    do {                                                                                                               \
        constexpr size_t lds = (size_t)gate_threads(L) * EPL * sizeof(float);                                             \
        hipLaunchKernelGGL((k_gate_grad<TT, L, EPL>), dim3(nblk), dim3(gate_threads(L)), lds, s, (const TT*)logits, T,    \
                           (int)E, (int)top, normalize, experts, counts, gweights, gloss, (TT*)out);                   \
    } while (0)
    if (xt == DType::F32) KM_GATE(float);
    else if (xt == DType::F16) KM_GATE(_Float16);
    else KM_GATE(uint16_t);
#undef KM_GO
    e = hipGetLastError();
    return e;
}

}  // namespace km

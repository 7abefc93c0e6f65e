// The gate of a layer of experts: the softmax of every token's logits, its
// largest ones in order, the choices counted, the loss that balances the
// experts, and the gradient of all of it.
//
// A row of E logits is held by a group of L lanes (16 up to 256 experts, so that
// every exchange is a DPP move inside 16 lanes; 64 beyond), expert j L + lane in
// register j.  Choosing is `top` rounds of two reductions: the largest key of
// the group, then the lowest expert that has it.
#include "codes8.h"

namespace km {

constexpr int kGateThreads = 256, kGateTopMax = 64;
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

// z[j] = exp(l[j] - m), m the largest logit that is a number; returns 1 / sum z
// (0 for a row of -infinity; NaN where a logit is NaN or +infinity).
template <int L, int EPL>
__device__ __forceinline__ float gate_softmax(const float (&l)[EPL], const uint32_t (&key)[EPL], float (&z)[EPL],
                                              float* m_out) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) top = top > key[j] ? top : key[j];
    top = lane_max<L>(top);
    const float m = top ? gate_value(top) : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        z[j] = expf(l[j] - m);
        sum += z[j];
    }
    sum = lane_sum<L>(sum);
    *m_out = m;
    return sum == 0.f ? 0.f : 1.f / sum;
}

// Blocks of the gate leave their counts and probabilities' sums: part_n[b][E + 1]
// (the last one: rows that are not all -infinity) and part_p[b][E].
template <typename T, int L, int EPL>
__global__ __launch_bounds__(kGateThreads) void k_gate(const T* __restrict__ logits, int64_t Tn, int E, int top,
                                                       bool normalize, int32_t* __restrict__ experts,
                                                       float* __restrict__ weights, int32_t* __restrict__ part_n,
                                                       float* __restrict__ part_p) {
    constexpr int G = kGateThreads / L, KR = kGateTopMax / L, GW = 64 / L;
    extern __shared__ int32_t s_cnt[];  // [E + 1]; then float [4][E]
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    for (int j = tid; j <= E; j += kGateThreads) s_cnt[j] = 0;
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
        const float inv = gate_softmax<L, EPL>(l, key, z, &m);
        if (inv != 0.f) {
            rows += lane == 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] = fmaf(z[j], inv, acc[j]);
        }
        float zk[KR], sum = 0.f;  // the choice k of lane k % L (-1: none)
#pragma unroll
        for (int u = 0; u < KR; ++u) zk[u] = -1.f;
        for (int k = 0; k < top; ++k) {
            uint32_t best = 0, at = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                if (key[j] > best) best = key[j], at = j;
            }
            const uint32_t most = lane_max<L>(best);
            const uint32_t e = lane_min<L>(best == most && most ? at * L + lane : 0xffffffffu);
            if (e % L == (uint32_t)lane && most) {
#pragma unroll
                for (int j = 0; j < EPL; ++j) key[j] = e / L == (uint32_t)j ? 0u : key[j];
                atomicAdd(&s_cnt[e], 1);
            }
            const float v = most ? expf(gate_value(most) - m) : -1.f;
            sum += most ? v : 0.f;
#pragma unroll
            for (int u = 0; u < KR; ++u) zk[u] = k == u * L + lane ? v : zk[u];
            if (in && lane == 0) experts[t * top + k] = most ? (int32_t)e : -1;
        }
        const float by = !normalize ? inv : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            const int k = u * L + lane;
            if (in && k < top) weights[t * top + k] = zk[u] < 0.f ? 0.f : zk[u] * by;
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
    int32_t* pn = part_n + (int64_t)blockIdx.x * (E + 1);
    float* pp = part_p + (int64_t)blockIdx.x * E;
    for (int e = tid; e <= E; e += kGateThreads) {
        pn[e] = s_cnt[e];
        if (e < E) pp[e] = ((s_p[e] + s_p[E + e]) + s_p[2 * E + e]) + s_p[3 * E + e];
    }
}

// Counts and shares of the blocks' parts, and the loss: one block.
__global__ __launch_bounds__(1024) void k_gate_fold(const int32_t* __restrict__ part_n, const float* __restrict__ part_p,
                                                    int nblk, int E, int32_t* __restrict__ counts,
                                                    float* __restrict__ shares, float* __restrict__ loss) {
    __shared__ float s_f[1024];
    __shared__ int64_t s_n[1024];
    const int tid = threadIdx.x;
    int32_t n = 0;
    for (int b = 0; b < nblk; ++b) n += part_n[(int64_t)b * (E + 1) + E];
    const float inv = n ? 1.f / (float)n : 0.f;
    float dot = 0.f;
    int64_t all = 0;
    for (int e = tid; e < E; e += 1024) {
        int32_t c = 0;
        float p = 0.f;
        for (int b = 0; b < nblk; ++b) {
            c += part_n[(int64_t)b * (E + 1) + e];
            p += part_p[(int64_t)b * E + e];
        }
        p *= inv;
        counts[e] = c;
        shares[e] = p;
        all += c;
        dot = fmaf((float)c, p, dot);
    }
    s_f[tid] = dot;
    s_n[tid] = all;
    __syncthreads();
    for (int o = 512; o >= 1; o >>= 1) {
        if (tid < o) s_f[tid] += s_f[tid + o], s_n[tid] += s_n[tid + o];
        __syncthreads();
    }
    if (tid == 0) {
        counts[E] = n;
        // (NaN shares make a NaN loss, also where no expert could be chosen)
        loss[0] = s_n[0] ? s_f[0] * (float)E / (float)s_n[0] : s_f[0] * 0.f;
    }
}

static int64_t gate_blocks(int64_t T, int64_t E) {
    const int64_t rows = E <= 256 ? kGateThreads / 16 : kGateThreads / 64, n = (T + rows - 1) / rows;
    return n < 1 ? 1 : n < 256 ? n : 256;
}
size_t gate_scratch(int64_t T, int64_t E) {
    return ((size_t)gate_blocks(T, E) * (2 * E + 1) * sizeof(int32_t) + 255) & ~(size_t)255;
}

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
    int32_t* pn = (int32_t*)ws;
    float* pp = (float*)(pn + nblk * (E + 1));
    const size_t lds = (size_t)(5 * E + 1) * sizeof(int32_t);
    hipError_t e = hipSuccess;
#define KM_GO(TT, L, EPL)                                                                                             \
    do {                                                                                                              \
        if (lds > 64 * 1024 && (e = hipFuncSetAttribute((const void*)k_gate<TT, L, EPL>,                              \
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)) != hipSuccess) \
            return e;                                                                                                 \
        hipLaunchKernelGGL((k_gate<TT, L, EPL>), dim3((unsigned)nblk), dim3(kGateThreads), lds, s, (const TT*)logits, \
                           T, (int)E, (int)top, normalize, experts, weights, pn, pp);                                 \
    } while (0)
    if (xt == DType::F32) KM_GATE(float);
    else if (xt == DType::F16) KM_GATE(_Float16);
    else KM_GATE(uint16_t);
#undef KM_GO
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_gate_fold, dim3(1), dim3(1024), 0, s, pn, pp, (int)nblk, (int)E, counts, shares, loss);
    return hipGetLastError();
}

// The gradient.  The chosen experts' part reaches the lane that owns the expert
// through LDS: a group writes its row, the lanes of the choices add to it, the
// group reads it back.
template <typename T, int L, int EPL>
__global__ __launch_bounds__(kGateThreads) void k_gate_grad(const T* __restrict__ logits, int64_t Tn, int E, int top,
                                                            bool normalize, const int32_t* __restrict__ experts,
                                                            const int32_t* __restrict__ counts,
                                                            const float* __restrict__ gweights,
                                                            const float* __restrict__ gloss, T* __restrict__ out) {
    constexpr int G = kGateThreads / L, KR = kGateTopMax / L;
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
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * L + lane;
            l[j] = in && e < E ? load_logit(logits + t * E + e) : -INFINITY;
            key[j] = gate_key(l[j]);
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
        const float inv = gate_softmax<L, EPL>(l, key, z, &m);
        // the choices' softmax numerators, and <w, gw> over the chosen
        float wk[KR], sum = 0.f, dot = 0.f;
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            wk[u] = ek[u] >= 0 ? expf(lk[u] - m) : 0.f;
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
    const int64_t rows = E <= 256 ? kGateThreads / 16 : kGateThreads / 64, n = (T + rows - 1) / rows;
    const unsigned nblk = (unsigned)(n < 2048 ? n : 2048);
    hipError_t e = hipSuccess;
#define KM_GO(TT, L, EPL)                                                                                              \
    do {                                                                                                               \
        constexpr size_t lds = (size_t)kGateThreads * EPL * sizeof(float);                                             \
        hipLaunchKernelGGL((k_gate_grad<TT, L, EPL>), dim3(nblk), dim3(kGateThreads), lds, s, (const TT*)logits, T,    \
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

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

// 16 bytes moved down by `by` (0 .. 16), zeros behind them.
__device__ __forceinline__ u32x4 move_down(u32x4 t, int by) {
    const int words = by >> 2, bits = (by & 3) * 8;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int j = i; j < 4; ++j) {
            lo = i + words == j ? t[j] : lo;
            hi = i + words + 1 == j ? t[j] : hi;
        }
        v[i] = (uint32_t)(((uint64_t)hi << 32 | lo) >> bits);
    }
    return v;
}

// 16 codes of a row of `len` at p, of which p[i], i < n, are in the row (n may be
// negative): the others as zeros.
__device__ __forceinline__ u32x4 load16_end(const uint8_t* __restrict__ p, int n, int64_t len) {
    if (n >= 16) return *(const u32x4_byte*)p;
    u32x4 v{0, 0, 0, 0};
    if (n <= 0) return v;
    if (len >= 16) return move_down(*(const u32x4_byte*)(p + n - 16), 16 - n);  // the row's last 16
#pragma nounroll
    for (int i = 0; i < n; ++i) {
        const uint32_t c = (uint32_t)p[i] << (8 * (i & 3));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] |= i >> 2 == j ? c : 0u;
    }
    return v;
}

// The same without branches, of a row that has 16 codes at least.
__device__ __forceinline__ u32x4 load16_in(const uint8_t* __restrict__ p, int n) {
    const int by = n >= 16 ? 0 : 16 - n;
    return move_down(*(const u32x4_byte*)(p - by), by < 16 ? by : 16);
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
            const int left = (int)(inner - i0 < 32 ? inner - i0 : 32);  // (negative: none)
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
                a[0] = load16_end(wm + o * K + i0, left, K);
                a[1] = load16_end(wm + o * K + i0 + 16, left - 16, K);
            }
            const float sw = GRAD ? ws[b * kb + ob] : ws[ob * kb + b];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint8_t* p = x + src[n] * inner + i0;
                const int have = src[n] < 0 ? 0 : left;
                const u32x4 x0 = load16_end(p, have, inner), x1 = load16_end(p + 16, have - 16, inner);
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

// Many rows.  The same product on blocks of 256 rows of the matrix (GRAD: its
// columns) and 16 NT tokens; each of four waves has 64 of the rows and all of the
// tokens.
//
// A step takes 128 of the inner length.  What it needs, codes of the matrix and of
// the tokens and their scales, comes to LDS by direct loads ST - 1 steps ahead.
// Rows of 128 codes are XOR-swizzled by 16-byte chunks.  (Operands straight from
// memory, 16 rows to an instruction, cost the texture path an access a lane: 217 us
// for the case below.)  GRAD wants columns of the matrix: a wave brings 128 rows by
// 64 columns and reads them transposed (ds_read_b64_tr_b8: a lane receives one
// column of eight rows).
//
// A wave runs alone on its SIMD, so nothing else hides its latencies: between the matrix instructions of a step stand the reads of the next
// step's operands from LDS, the direct loads of a later one, and the scaling of
// the results of two instructions before.
//
// DIRECT: rows of x and of the matrix start at 16-byte boundaries; otherwise codes
// are copied through registers.
constexpr int kTileWaves = 4, kTileThreads = 64 * kTileWaves, kTileRows = 64 * kTileWaves;

constexpr int kTileStages = 3;

template <int NT>
struct BlockTile {
    static constexpr int TT = 16 * NT;
    static constexpr int X = TT * kBlock8, W = kTileRows * kBlock8;  // codes of a step
    static constexpr int SX = X + W;                                 // the tokens' scales: [16][NT]
    static constexpr int SW = SX + (TT < 64 ? 64 : TT) * 4;          // the wave's block's scale, 64 times
    static constexpr int STAGE = SW + kTileWaves * 256;
    static constexpr int BYTES = kTileStages * STAGE;
    static constexpr int LOADS = TT / 32 + 8 + 2;                    // a wave's direct loads of a step
};

// 16-byte chunk of row m (of 64 columns) that holds columns 16 c .. 16 c + 15: the
// 32 rows that a transposing read touches spread over all banks.
__device__ __forceinline__ int tile_chunk(int c, int m) { return c ^ ((m >> 2 & 1) ^ (m >> 4 & 3)); }

// What direct loads of codes behind a row's end read.
__device__ const u32x4 g_no_codes = {0, 0, 0, 0};

template <int V>
struct Int {
    static constexpr int value = V;
};

template <typename O, int NT, bool GRAD, bool DIRECT>
__global__ __launch_bounds__(kTileThreads, 1) void k_block_tile(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t S, const uint8_t* __restrict__ codes,
    const float* __restrict__ scales, int E, int64_t M, int64_t K, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ order, int64_t top, O* __restrict__ out) {
    typedef BlockTile<NT> L;
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    constexpr int TT = L::TT, ST = kTileStages, R = 4, NX = TT / 32, NW = 8, NI = NT * R;
    static_assert(NT % 2 == 0 && TT <= 128, "32 tokens to an instruction of every wave, scales by two waves");
    extern __shared__ __attribute__((aligned(16))) char s_mem[];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const Segment g = find_segment(offsets, S, E, TT, blockIdx.y);
    if (g.e < 0) return;
    const int64_t inner = GRAD ? M : K, outer = GRAD ? K : M, ib = blocks8(inner), kb = blocks8(K);
    const int64_t o0 = (int64_t)blockIdx.x * kTileRows + w * 64;  // the wave's rows
    f32x4 acc[R][NT];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[a][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint32_t none = 0;  // bit n: token n 16 + r is a row of none
    if (g.e < E) {
        const uint8_t* wm = codes + (int64_t)g.e * M * K;
        const float* ws = scales + (int64_t)g.e * blocks8(M) * kb;
        auto source = [&](int t) { return source_row(order, top, S, g.p0 + (t < g.n ? t : g.n - 1)); };
        // A thread's chunks of tokens: 8 a token, chunk (lane & 7) ^ token at place lane & 7, as
        // 32-bit offsets from the segment's first row (with an order: from x's, whose rows are
        // less than 4 GB then).
        const uint8_t* xb = order ? x : x + g.p0 * inner;
        uint32_t xo[NX];
        const int xc = ((tid & 7) ^ (tid >> 3 & 7)) * 16;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int64_t src = source((i * kTileThreads + tid) >> 3);
            xo[i] = (uint32_t)((order ? (src < 0 ? 0 : src) : src - g.p0) * inner) + xc;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) none |= (order && source(n * 16 + r) < 0 ? 1u : 0u) << n;
        // the token whose scale this lane fetches: place p of [16][NT]
        const float* xsp;
        {
            int p = TT > 64 ? (w & 1) * 64 + lane : lane;
            p = p < TT ? p : TT - 1;
            const int64_t src = source(p % NT * 16 + p / NT);
            xsp = xs + (src < 0 ? 0 : src) * ib;
        }
        const int64_t ob = (o0 < outer ? o0 : outer - 1) / kBlock8;
        // Of the matrix, forward: rows of the wave like the tokens' (it reads no others'); GRAD:
        // 16 rows of 64 columns an instruction, place lane & 3 of row m holding chunk
        // tile_chunk(lane & 3, m).  Rows behind the last one read it.
        const uint8_t* wb = wm + (GRAD ? 0 : (o0 < outer ? o0 : outer - 1) * K);
        uint32_t wo[NW];
        const int wrow = GRAD ? lane >> 2 : lane >> 3;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if constexpr (GRAD) {
                const int64_t col = o0 + tile_chunk(lane & 3, i * 16 + wrow) * 16;
                wo[i] = (uint32_t)((i * 16 + wrow) * K) + (uint32_t)(col < outer ? col : 0);
            } else {
                const int64_t left = outer - 1 - o0, row = i * 8 + wrow;
                wo[i] = (uint32_t)((row < left ? row : left < 0 ? 0 : left) * K) + ((lane & 7) ^ (lane >> 3)) * 16;
            }
        }
        auto wbase = [&](int64_t st) { return wb + st * kBlock8 * (GRAD ? K : 1); };
        auto to_x = [&](int stage, int i) { return s_mem + stage * L::STAGE + (i * kTileThreads + w * 64) * 16; };
        auto to_w = [&](int stage, int i) { return s_mem + stage * L::STAGE + L::X + w * (64 * kBlock8) + i * 1024; };
        // direct load i of step st; LAST: of a step that the inner length ends in
        auto load = [&](int64_t st, int stage, int i, auto last_tag) {
            constexpr bool LAST = decltype(last_tag)::value;
            const int left = (int)(inner - st * kBlock8);
            if (i < NX) {
                if constexpr (!DIRECT) return;
                const uint8_t* b = xb + st * kBlock8;
                if constexpr (LAST) dma16_lane(xc < left ? (const void*)(b + xo[i]) : (const void*)&g_no_codes, to_x(stage, i));
                else dma16((const char*)b, xo[i], to_x(stage, i));
            } else if (i < NX + NW) {
                if constexpr (!DIRECT) return;
                const int u = i - NX;
                const uint8_t* b = wbase(st);
                if constexpr (!LAST) {
                    dma16((const char*)b, wo[u], to_w(stage, u));
                } else if constexpr (GRAD) {
                    // (rows behind the last one meet zeros of x)
                    const int m = u * 16 + wrow;
                    dma16_lane(b + wo[u] - (m < left ? 0 : (int64_t)(m - left + 1) * K), to_w(stage, u));
                } else {
                    dma16_lane(((lane & 7) ^ (lane >> 3)) * 16 < left ? (const void*)(b + wo[u]) : (const void*)&g_no_codes,
                               to_w(stage, u));
                }
            } else if (i == NX + NW) {
                dma4_lane(xsp + st, s_mem + stage * L::STAGE + L::SX + (TT > 64 ? (w & 1) * 256 : 0));
            } else {
                dma4_lane(GRAD ? ws + st * kb + ob : ws + ob * kb + st, s_mem + stage * L::STAGE + L::SW + w * 256);
            }
        };
        // the same through registers: codes only
        struct Copy {
            u32x4 x[NX], w[NW];
        };
        auto copy = [&](int64_t st, Copy& c, auto last_tag) {
            constexpr bool LAST = decltype(last_tag)::value;
            const int left = (int)(inner - st * kBlock8 < kBlock8 ? inner - st * kBlock8 : kBlock8);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const uint8_t* p = xb + st * kBlock8 + xo[i];
                c.x[i] = LAST ? load16_in(p, left - xc) : *(const u32x4_byte*)p;
            }
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const uint8_t* p = wbase(st) + wo[i];
                if constexpr (!LAST) {
                    c.w[i] = *(const u32x4_byte*)p;
                } else if constexpr (GRAD) {
                    // columns behind the row's end hold the next row's and give results that are not
                    // stored; nothing behind the matrix is read
                    const int m = i * 16 + wrow;
                    p -= m < left ? 0 : (int64_t)(m - left + 1) * K;
                    c.w[i] = load16_in(p, (int)(wm + M * K - p < 16 ? wm + M * K - p : 16));
                } else {
                    c.w[i] = load16_in(p, left - ((lane & 7) ^ (lane >> 3)) * 16);
                }
            }
        };
        auto keep = [&](int stage, const Copy& c) {
#pragma unroll
            for (int i = 0; i < NX; ++i) *(u32x4*)(to_x(stage, i) + lane * 16) = c.x[i];
#pragma unroll
            for (int i = 0; i < NW; ++i) *(u32x4*)(to_w(stage, i) + lane * 16) = c.w[i];
        };
        auto fill = [&](int64_t st, int stage) {  // the whole step
            st = st < ib ? st : ib - 1;
#pragma unroll
            for (int i = 0; i < L::LOADS; ++i) load(st, stage, i, Int<1>{});
            if constexpr (!DIRECT) {
                Copy c;
                copy(st, c, Int<1>{});
                keep(stage, c);
            }
        };
        // operands of a step from its stage
        auto matrix = [&](int stage, int a) {
            const char* wl = s_mem + stage * L::STAGE + L::X + w * (64 * kBlock8);
            if constexpr (GRAD) {
                // rows q 16 + (0 .. 15) and 64 more of column a 16 + r: a lane fetches 8 bytes of
                // row r / 2 of eight, half r % 2 of the chunk
                i32x8 v;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int m = (f >> 1) * 64 + q * 16 + (f & 1) * 8 + (r >> 1);
                    const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (__attribute__((address_space(3))) i32x2*)(wl + m * 64 + tile_chunk(a, m) * 16 + (r & 1) * 8));
                    v[2 * f] = t[0];
                    v[2 * f + 1] = t[1];
                }
                return v;
            } else {
                const char* row = wl + (a * 16 + r) * kBlock8;
                return join8(*(const u32x4*)(row + ((q ^ (r & 7)) * 16)), *(const u32x4*)(row + (((q + 4) ^ (r & 7)) * 16)));
            }
        };
        auto tokens = [&](int stage, int n) {
            const char* row = s_mem + stage * L::STAGE + (n * 16 + r) * kBlock8;
            return join8(*(const u32x4*)(row + ((q ^ (r & 7)) * 16)), *(const u32x4*)(row + (((q + 4) ^ (r & 7)) * 16)));
        };
        struct Step {
            i32x8 a[R], b[NT];
            float sx[NT], sw;
        };
        auto read_scales = [&](int stage, Step& f) {
            const float* sx = (const float*)(s_mem + stage * L::STAGE + L::SX) + r * NT;
#pragma unroll
            for (int n = 0; n < NT; ++n) f.sx[n] = sx[n];
            f.sw = ((const float*)(s_mem + stage * L::STAGE + L::SW))[w * 64 + lane];
        };
        // One barrier a step: before it, this wave's loads of the next step have landed (those of
        // later ones are still on their way) and its reads of this step are done.
        auto landed = [&](auto ahead_tag) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(DIRECT ? vmcnt_imm(decltype(ahead_tag)::value * L::LOADS) & ~(15u << 8) : 0);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        };
        Step f[2];
        // part k of a step's operands: scales, rows, tokens
        constexpr int PARTS = 1 + R + NT;
        auto read = [&](int stage, Step& s, int k) {
            if (k == 0) read_scales(stage, s);
            else if (k <= R) s.a[k - 1] = matrix(stage, k - 1);
            else s.b[k - 1 - R] = tokens(stage, k - 1 - R);
        };
        int now = 0, next = 1;  // stages of this step and the next
        auto step = [&](int64_t st, auto c_tag, auto last_tag) {
            constexpr int c = decltype(c_tag)::value;
            landed(Int<ST - 2>{});
            const int64_t far = st + ST < ib ? st + ST : ib - 1;
            Copy cp;
            if constexpr (!DIRECT) copy(far, cp, last_tag);
            f32x4 d[3];
#pragma unroll
            for (int i = 0; i < NI + 2; ++i) {
                if (i < NI) d[i % 3] = mfma8(f[c].a[i % R], f[c].b[i / R], f32x4{0.f, 0.f, 0.f, 0.f});
                __builtin_amdgcn_sched_barrier(0);
                // the next step's operands and the direct loads of a later one, spread over this
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
                    if (i == 1 + k * (NI - 3) / PARTS) read(next, f[c ^ 1], k);
#pragma unroll
                for (int k = 0; k < L::LOADS; ++k)
                    if (i == k * (NI - 1) / L::LOADS) load(far, now, k, last_tag);
                __builtin_amdgcn_sched_barrier(0);
                if (i >= 2) {
                    const int n = (i - 2) / R, a = (i - 2) % R;
                    if (a == 0) f[c].sx[n] *= f[c].sw;
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[a][n][e] = fmaf(f[c].sx[n], d[(i - 2) % 3][e], acc[a][n][e]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (!DIRECT) keep(now, cp);
            now = next;
            next = next + 1 == ST ? 0 : next + 1;
        };
#pragma unroll
        for (int i = 0; i < ST; ++i) fill(i, i);
        landed(Int<ST - 1>{});
#pragma unroll
        for (int k = 0; k < PARTS; ++k) read(0, f[0], k);
        // steps during which no loads of the last one begin, then the others
        int64_t st = 0;
        for (; st + 1 + ST < ib - 1; st += 2) {
            step(st, Int<0>{}, Int<0>{});
            step(st + 1, Int<1>{}, Int<0>{});
        }
        for (; st + 1 < ib; st += 2) {
            step(st, Int<0>{}, Int<1>{});
            step(st + 1, Int<1>{}, Int<1>{});
        }
        if (st < ib) step(st, Int<0>{}, Int<1>{});
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // (nothing writes to LDS behind the block's end)
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = n * 16 + r;
        if (t >= g.n) continue;
        const bool no = none >> n & 1;
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const int64_t o = o0 + a * 16 + q * 4;
            if (o < outer)
                store_results<O>(out + (g.p0 + t) * outer + o, outer - o, no ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[a][n]);
        }
    }
}

size_t block_product_scratch(int64_t, int64_t, int64_t, int64_t) { return 0; }
size_t block_product_grad_scratch(int64_t, int64_t, int64_t, int64_t) { return 0; }

template <typename O, bool GRAD>
static hipError_t block_launch(const BlockArgs& a, hipStream_t s) {
    const int64_t inner = GRAD ? a.M : a.K, outer = GRAD ? a.K : a.M;
    const bool direct = inner % 16 == 0 && (uintptr_t)a.x % 16 == 0 && (!GRAD || (a.K % 16 == 0 && (uintptr_t)a.codes % 16 == 0));
    hipError_t e = hipSuccess;
#define KM_ARGS                                                                                                        \
    (const uint8_t*)a.x, a.x_scales, a.S, (const uint8_t*)a.codes, a.scales, (int)a.E, a.M, a.K, a.offsets, a.order,   \
        a.top, (O*)a.out
#define KM_GO2(NT, DIR)                                                                                                \
    do {                                                                                                               \
        constexpr int lds = BlockTile<NT>::BYTES;                                                                      \
        if ((e = hipFuncSetAttribute((const void*)k_block_tile<O, NT, GRAD, DIR>,                                      \
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds)) != hipSuccess)                  \
            return e;                                                                                                  \
        hipLaunchKernelGGL((k_block_tile<O, NT, GRAD, DIR>),                                                           \
                           dim3((unsigned)((outer + kTileRows - 1) / kTileRows),                                       \
                                (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * NT)),                                \
                           dim3(kTileThreads), lds, s, KM_ARGS);                                                       \
    } while (0)
#define KM_GO(NT)                      \
    do {                               \
        if (direct) KM_GO2(NT, true);  \
        else KM_GO2(NT, false);        \
    } while (0)
    // (copies through registers take 16 codes of a row, or of a matrix, at least)
    if (a.S >= 32 * a.E && inner >= 16 && a.M * a.K >= 16) {
        KM_GO(8);
        return hipGetLastError();
    }
#undef KM_GO
#undef KM_GO2
    hipLaunchKernelGGL((k_block_few<O, 8, 1, GRAD>),
                       dim3((unsigned)((outer + 15) / 16), (unsigned)segment_tiles(a.S, a.E, a.offsets, 16)), dim3(512),
                       0, s, KM_ARGS);
#undef KM_ARGS
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

// Products of 8-bit rows with 8-bit matrices that have a float32 scale for each
// block of 128 x 128, one matrix per expert, and the gradient of their input.
#include "block_copy.h"
#include "codes.h"
#include "codes8.h"

namespace km {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// D = A B on a block of 128: 16 x 16 results, lane (r, q) holding 32 codes of
// row r of A and of column r of B (any order of the 128, the same in both).
// (Its sums keep 13 bits below the largest of eight products; four instructions of 32
// codes give the same bits in 1.4 times the time.)
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

// 16 codes of a row of 16 at least at p, of which p[i], i < n, are in the row (n may
// be negative): the others as zeros, without branches.
__device__ __forceinline__ u32x4 load16_in(const uint8_t* __restrict__ p, int n) {
    const int by = tile_back(n);
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

// Inner lengths below 16 codes, too short for the other kernels' copies of 16 bytes:
// out = W x^T, one 16 x 16 x 128 instruction for 16 rows of the matrix (as A; GRAD:
// its columns) and 16 tokens, a wave each.  The lanes of the first 16 codes read them
// byte by byte; the others hold zeros.
template <typename O, bool GRAD>
__global__ __launch_bounds__(64) void k_block_short(const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t S,
                                                    const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                                                    int E, int64_t M, int64_t K, const int32_t* __restrict__ offsets,
                                                    const int32_t* __restrict__ order, int64_t top, int64_t y0,
                                                    O* __restrict__ out) {
    const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
    const Segment g = find_segment(offsets, S, E, 16, (int)(y0 + blockIdx.y));
    if (g.e < 0) return;
    const int64_t outer = GRAD ? K : M, o0 = (int64_t)blockIdx.x * 16;
    const int inner = (int)(GRAD ? M : K);
    f32x4 v{0.f, 0.f, 0.f, 0.f};
    if (g.e < E) {
        const int64_t src = source_row(order, top, S, g.p0 + (r < g.n ? r : g.n - 1));
        const int64_t o = o0 + r < outer ? o0 + r : outer - 1;
        const uint8_t* wp = codes + (int64_t)g.e * M * K + (GRAD ? o : o * K);
        const uint8_t* xp = x + (src < 0 ? 0 : src) * inner;
        const int64_t step = GRAD ? K : 1;
        u32x4 a{0, 0, 0, 0}, b{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 15; ++j)
            if (q == 0 && j < inner) {
                a[j / 4] |= (uint32_t)wp[j * step] << (8 * (j % 4));
                b[j / 4] |= (uint32_t)xp[j] << (8 * (j % 4));
            }
        // (one block of the inner length)
        const float s = scales[(int64_t)g.e * blocks8(outer) + o0 / kBlock8] * xs[src < 0 ? 0 : src];
        const u32x4 no{0, 0, 0, 0};
        const f32x4 d = mfma8(join8(a, no), join8(b, no), f32x4{0.f, 0.f, 0.f, 0.f});
        if (src >= 0) {  // (codes and scales that are no numbers stay out of a row of none)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = s * d[i];
        }
    }
    const int64_t o = o0 + q * 4;
    if (r < g.n && o < outer) store_results<O>(out + (g.p0 + r) * outer + o, outer - o, v);
}

// Many rows.  The same product on blocks of 256 rows of the matrix (GRAD: its
// columns) and 16 NT tokens; each of its four waves has 64 of the rows and all of
// the tokens.
//
// A step takes 128 of the inner length.  What it needs, codes of the matrix and of
// the tokens and their scales, comes to LDS by direct loads ST - 1 steps ahead.
// Rows of 128 codes are XOR-swizzled by 16-byte chunks.  (Operands straight from
// memory, 16 rows to an instruction, cost the texture path an access a lane: 217 us
// for the case below.)  GRAD wants columns of the matrix: a wave brings 128 rows by
// 64 columns and reads them transposed (ds_read_b64_tr_b8: a lane receives one
// column of eight rows).
//
// A wave runs alone on its SIMD, so nothing else hides its latencies: between the
// matrix instructions of a step stand the reads of the next step's operands from
// LDS, the direct loads of a later one, and the scaling of the results of two
// instructions before.
//
// DIRECT: rows of x and of the matrix start at 16-byte boundaries; otherwise codes
// are copied through registers.
constexpr int kTileThreads = 256, kTileRows = 256;

template <int NT>
struct BlockTile {
    static constexpr int TT = 16 * NT;
    static constexpr int X = TT * kBlock8, W = kTileRows * kBlock8;  // codes of a step
    static constexpr int SX = X + W;                         // the tokens' scales: [16][NT]
    static constexpr int SW = SX + (TT + 63) / 64 * 256;     // the scale of each wave's rows, 64 times
    static constexpr int STAGE = SW + 4 * 256;
    static constexpr int SRC = kTileStages * STAGE;          // the tokens' rows of x
    static constexpr int BYTES = SRC + TT * 4;
    static constexpr int LOADS = NT / 2 + 8 + 2;             // a wave's direct loads of a step
};

// What direct loads of codes behind a row's end read.
__device__ const u32x4 g_no_codes = {0, 0, 0, 0};

template <typename O, int NT, bool GRAD, bool DIRECT>
__global__ __launch_bounds__(kTileThreads, 1) void k_block_tile(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t S, const uint8_t* __restrict__ codes,
    const float* __restrict__ scales, int E, int64_t M, int64_t K, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ order, int64_t top, int64_t steps_per, O* __restrict__ out, float* __restrict__ part) {
    typedef BlockTile<NT> L;
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    constexpr int TT = L::TT, ST = kTileStages, R = 4, NX = NT / 2, NW = 8, NI = NT * R;
    static_assert(NT % 2 == 0 && TT <= 128, "whole instructions of every wave, scales by two waves");
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
    int32_t* s_src = (int32_t*)(s_mem + L::SRC);  // -1: a row of none
    // the steps of this split of the inner length
    const int64_t s0 = blockIdx.z * steps_per, s1 = s0 + steps_per < ib ? s0 + steps_per : ib;
    if (g.e < E && s0 < s1) {
        const uint8_t* wm = codes + (int64_t)g.e * M * K;
        const float* ws = scales + (int64_t)g.e * blocks8(M) * kb;
        if (tid < TT) s_src[tid] = (int32_t)source_row(order, top, S, g.p0 + (tid < g.n ? tid : g.n - 1));
        __syncthreads();
        // a thread's chunks of tokens: 8 a token, chunk (lane & 7) ^ token at place lane & 7
        const int xc = ((tid & 7) ^ (tid >> 3 & 7)) * 16;
        // their rows of x (GRAD, whose rows follow each other: 32-bit offsets from the segment)
        const uint8_t* xb = GRAD ? x + g.p0 * inner : x;
        uint32_t xr[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int32_t src = s_src[(i * kTileThreads + tid) >> 3];
            xr[i] = GRAD ? (uint32_t)((src - g.p0) * inner) + xc : src < 0 ? 0 : src;
        }
        auto xp = [&](int64_t st, int i) {
            return xb + st * kBlock8 + (GRAD ? (uint64_t)xr[i] : xc + (uint64_t)xr[i] * (uint32_t)inner);
        };
        // the token whose scale this lane fetches: place p of [16][NT]
        const float* xsp;
        {
            int p = TT > 64 ? (w & 1) * 64 + lane : lane;
            p = p < TT ? p : TT - 1;
            const int64_t src = s_src[p % NT * 16 + p / NT];
            xsp = xs + (src < 0 ? 0 : src) * ib;
        }
        const int64_t ob = (o0 < outer ? o0 : outer - 1) / kBlock8;
        // Of the wave's rows of the matrix, instruction i.  Forward: 8 of them, like the tokens';
        // GRAD: 16 rows of 64 columns, place lane & 3 of row m holding chunk
        // tile_chunk(lane & 3, m).  Rows behind the last one read it.
        const uint8_t* wb = wm + (GRAD ? 0 : (o0 < outer ? o0 : outer - 1) * K);
        uint32_t wo[NW];
        const int wrow = GRAD ? lane >> 2 : lane >> 3;
#pragma unroll
        for (int i = 0; i < NW; ++i) wo[i] = tile_matrix_at(GRAD, K, outer, o0, i, lane);
        auto wbase = [&](int64_t st) { return wb + st * kBlock8 * (GRAD ? K : 1); };
        auto to_x = [&](int stage, int i) { return s_mem + stage * L::STAGE + (i * kTileThreads + w * 64) * 16; };
        auto to_w = [&](int stage, int i) { return s_mem + stage * L::STAGE + L::X + w * (64 * kBlock8) + i * 1024; };
        // direct load i of step st; LAST: of a step that may need bounds
        auto load = [&](int64_t st, int stage, int i, auto last_tag) {
            constexpr bool LAST = decltype(last_tag)::value;
            const int left = (int)(inner - st * kBlock8);
            if (i < NX) {
                if constexpr (!DIRECT) return;
                if constexpr (LAST) dma16_lane(xc < left ? (const void*)xp(st, i) : (const void*)&g_no_codes, to_x(stage, i));
                else if constexpr (GRAD) dma16((const char*)(xb + st * kBlock8), xr[i], to_x(stage, i));
                else dma16_lane(xp(st, i), to_x(stage, i));
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
                const uint8_t* p = xp(st, i);
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
            st = s0 + st < s1 ? s0 + st : s1 - 1;
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
            const int64_t far = st + ST < s1 ? st + ST : s1 - 1;
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
        // steps during which only loads without bounds begin, then the others
        int64_t st = s0;
        for (; st + 1 + ST < tile_free_end(s1, GRAD, DIRECT); st += 2) {
            step(st, Int<0>{}, Int<0>{});
            step(st + 1, Int<1>{}, Int<0>{});
        }
        for (; st + 1 < s1; st += 2) {
            step(st, Int<0>{}, Int<1>{});
            step(st + 1, Int<1>{}, Int<1>{});
        }
        if (st < s1) step(st, Int<0>{}, Int<1>{});
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // (nothing writes to LDS behind the block's end)
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = n * 16 + r;
        if (t >= g.n) continue;
        const bool no = g.e < E && s0 < s1 && s_src[t] < 0;
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const int64_t o = o0 + a * 16 + q * 4;
            if (o >= outer) continue;
            const f32x4 v = no ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[a][n];
            const int64_t at = (g.p0 + t) * outer + o;
            if (part) store_results<float>(part + blockIdx.z * S * outer + at, outer - o, v);
            else store_results<O>(out + at, outer - o, v);
        }
    }
}

// Few rows, aligned ones.  Each wave streams the columns of its own 16 R rows of
// the matrix, and those of 16 NT tokens, through three slots of LDS by direct loads
// of whole lines (straight to operands, 16 rows an instruction, the texture path
// takes an access a lane: 32 us for the case below).  A block's WR x WK waves are
// WR groups of rows; the WK waves of a group take every WK-th block of 128 columns,
// and their sums are added in LDS in order.  Waves meet only there.
constexpr int kStreamSlots = 3, kStreamScales = 8;

template <int WR, int WK, int R, int NT>
struct BlockStream {
    static constexpr int SLOT = (R + NT) * 16 * kBlock8, LOADS = (R + NT) * 2;
    static constexpr int RING = WR * WK * kStreamSlots * SLOT, SUMS = WK > 1 ? WR * WK * R * NT * 64 * 16 : 0;
    static constexpr int BYTES = RING > SUMS ? RING : SUMS;
};

template <typename O, int WR, int WK, int R, int NT>
__global__ __launch_bounds__(64 * WR * WK) void k_block_stream(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t S, const uint8_t* __restrict__ codes,
    const float* __restrict__ scales, int E, int64_t M, int64_t K, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ order, int64_t top, O* __restrict__ out) {
    typedef BlockStream<WR, WK, R, NT> L;
    constexpr int D = kStreamSlots, C = kStreamScales, TT = 16 * NT;
    extern __shared__ __attribute__((aligned(16))) char s_mem[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = w / WK, wk = w % WK, r = lane & 15, q = lane >> 4, row8 = lane >> 3;
    const int at = ((lane & 7) ^ row8) * 16;  // the lane's chunk of a row: place lane & 7 holds chunk (lane & 7) ^ row
    const Segment g = find_segment(offsets, S, E, TT, blockIdx.y);
    if (g.e < 0) return;
    const int64_t kb = blocks8(K), o0 = ((int64_t)blockIdx.x * WR + wr) * 16 * R;
    f32x4 acc[R][NT];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[a][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    bool none[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) none[n] = false;
    if (g.e < E) {
        const uint8_t* wm = codes + (int64_t)g.e * M * K + at;
        const uint8_t *wp[2 * R], *xp[2 * NT];
        const float* xsp[NT];
#pragma unroll
        for (int u = 0; u < 2 * R; ++u) {
            const int64_t o = o0 + u * 8 + row8;
            wp[u] = wm + (o < M ? o : M - 1) * K;
        }
        auto source = [&](int t) { return source_row(order, top, S, g.p0 + (t < g.n ? t : g.n - 1)); };
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) {
            const int64_t src = source(u * 8 + row8);
            xp[u] = x + (src < 0 ? 0 : src) * K + at;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t src = source(n * 16 + r);
            none[n] = src < 0;
            xsp[n] = xs + (src < 0 ? 0 : src) * kb;
        }
        const float* ws = scales + ((int64_t)g.e * blocks8(M) + (o0 < M ? o0 : M - 1) / kBlock8) * kb;
        char* ring = s_mem + w * (D * L::SLOT);
        const int64_t mine = wk < kb ? (kb - wk + WK - 1) / WK : 0;  // the wave's blocks: wk + WK i
        auto fill = [&](int64_t i, int slot) {
            const int64_t b = (wk + WK * i) * kBlock8;
            const bool in = b + at < K;  // (a row's last block may hold fewer codes)
#pragma unroll
            for (int u = 0; u < 2 * R; ++u)
                dma16_lane(in ? (const void*)(wp[u] + b) : (const void*)&g_no_codes, ring + slot * L::SLOT + u * 1024);
#pragma unroll
            for (int u = 0; u < 2 * NT; ++u)
                dma16_lane(in ? (const void*)(xp[u] + b) : (const void*)&g_no_codes, ring + slot * L::SLOT + (2 * R + u) * 1024);
        };
        auto operand = [&](int slot, int tile) {
            const char* row = ring + slot * L::SLOT + (tile * 16 + r) * kBlock8;
            return join8(*(const u32x4*)(row + ((q ^ (r & 7)) * 16)), *(const u32x4*)(row + (((q + 4) ^ (r & 7)) * 16)));
        };
        for (int64_t c0 = 0; c0 < mine; c0 += C) {
            const int n = mine - c0 < C ? (int)(mine - c0) : C;
            float sx[C][NT], sw[C];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int64_t b = wk + WK * (c0 + (i < n ? i : n - 1));
                sw[i] = ws[b];
#pragma unroll
                for (int t = 0; t < NT; ++t) sx[i][t] = xsp[t][b];
            }
#pragma unroll
            for (int i = 0; i < D; ++i)
                if (i < n) fill(c0 + i, i);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (i >= n) break;  // (uniform)
                const int slot = i % D;
                asm volatile("" ::: "memory");
                if (i + D <= n) __builtin_amdgcn_s_waitcnt(vmcnt_imm((D - 1) * L::LOADS));
                else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
                asm volatile("" ::: "memory");
                i32x8 av[R], bv[NT];
#pragma unroll
                for (int a = 0; a < R; ++a) av[a] = operand(slot, a);
#pragma unroll
                for (int t = 0; t < NT; ++t) bv[t] = operand(slot, R + t);
                asm volatile("" ::: "memory");
                __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(15u << 8));  // read, then filled again
                asm volatile("" ::: "memory");
                if (i + D < n) fill(c0 + i + D, slot);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float s = sw[i] * sx[i][t];
#pragma unroll
                    for (int a = 0; a < R; ++a) {
                        const f32x4 d = mfma8(av[a], bv[t], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[a][t][e] = fmaf(s, d[e], acc[a][t][e]);
                    }
                }
            }
        }
    }
    auto store = [&](int row, int a, int t, int l, f32x4 v) {
        const int tk = t * 16 + (l & 15);
        const int64_t o = ((int64_t)blockIdx.x * WR + row) * 16 * R + a * 16 + (l >> 4) * 4;
        if (tk < g.n && o < M) store_results<O>(out + (g.p0 + tk) * M + o, M - o, v);
    };
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (none[t]) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (WK == 1) store(wr, a, t, lane, acc[a][t]);
        }
    if constexpr (WK > 1) {
        __syncthreads();  // every wave is done with its slots
        f32x4* sums = (f32x4*)s_mem;  // [WR][WK][R][NT][64]
        constexpr int PER = R * NT * 64;
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int t = 0; t < NT; ++t) sums[((w * R + a) * NT + t) * 64 + lane] = acc[a][t];
        __syncthreads();
        for (int i = threadIdx.x; i < WR * PER; i += 64 * WR * WK) {
            const int row = i / PER, rest = i % PER;
            f32x4 v = sums[row * WK * PER + rest];
#pragma unroll
            for (int k = 1; k < WK; ++k) v += sums[(row * WK + k) * PER + rest];
            store(row, rest / (64 * NT), rest / 64 % NT, rest & 63, v);
        }
    }
}

// out[i] = the sum of nsplit partial sums, in order; four elements a thread.
template <typename O>
__global__ __launch_bounds__(256) void k_block_join(const float* __restrict__ part, int64_t n, int nsplit,
                                                    O* __restrict__ out, int64_t block0) {
    typedef f32x4 f32x4_any __attribute__((aligned(4)));
    const int64_t i = ((block0 + blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    if (i + 4 <= n) {
        f32x4 a = *(const f32x4_any*)(part + i);
        for (int s = 1; s < nsplit; ++s) a += *(const f32x4_any*)(part + s * n + i);
        store_results<O>(out + i, 4, a);
    } else {
        for (int64_t j = i; j < n; ++j) {
            float a = part[j];
            for (int s = 1; s < nsplit; ++s) a += part[s * n + j];
            out[j] = elem_from<O>(a);
        }
    }
}

// How a product is launched: token tiles of a block (0: not the kernel of many rows)
// and splits of the inner length, or the waves of a group in the kernel of few
// aligned rows (0: not that one), by the time each would take, us:
//   many rows   rounds of 256 blocks (one for each compute unit) of (steps of a
//               split x step + 4), a step 0.46, 0.6, 0.78, 0.95 for 2, 4, 6, 8 token
//               tiles and at least 1.05 where the matrices come from memory (64 MB or
//               more); splits add 4 and their sums' way through memory
//   few rows    3 + the matrices once for every 16 tokens at 11 TB/s, a fifth more
//               where an expert has several such tiles
//   both        no less than the matrices take from memory, 5.1 TB/s
// Where the matrices come from memory, tiles of 64, 96 and 128 tokens tie in the model
// as long as their rounds do, and the smallest is taken.  Measured (bf16, us a call in
// a graph that repeats it, so that matrices of up to 256 MB are in the memory-side
// cache; s8 .. s1: the kernel of few rows with 8 .. 1 waves a group; token tiles /
// splits; last what this function chooses):
//   rows, matrices                s8     s4     s2     s1    2/1    2/2    4/1    4/2    6/1    8/1    8/2  rule
//       1, 4096 x 4096           5.2    6.4    8.6   13.4   17.4   12.5   20.2   14.4   24.3   29.6   19.6  s8
//      64, 4096 x 4096          20.1    9.9    9.9   15.4   17.7   14.2   21.8   16.8   25.8   30.8   21.9  s4
//     256, 4096 x 4096          72.4   29.6   25.3   22.8   17.9   19.0   21.9   21.3   26.7   33.0   28.2  2/1
//    1024, 4096 x 4096         282.2  103.4   90.2   82.9   35.7   52.2   26.5   42.0   31.1   35.7   34.6  4/1
//    4096, 4096 x 4096          1119  397.4  348.7  317.1  136.5  192.4   98.9  148.0   94.5   84.2  126.9  8/1
//      64, 16 of 4096 x 2048    63.0   28.5   25.5   24.5   23.9   29.2   24.2   29.8   24.7   31.7   33.4  s1
//     128, 8 of 4096 x 4096     63.5   31.3   28.9   29.2   24.7   27.6   25.2   28.0   27.2   31.9   31.1  s2
//     512, 8 of 4096 x 4096    189.6   73.9   62.0   60.3   38.8   43.1   30.8   41.5   30.3   34.0   36.0  4/1
//    4096, 8 of 4096 x 4096     1341  469.5  371.7  336.4  161.6  293.0  124.0  206.0  101.7  111.8  159.3  6/1
//    8192, 8 of 4096 x 4096     2661  924.1  720.3  650.5  304.4  535.6  218.5  413.9  188.9  189.2  316.1  8/1
//      64, 128 of 2048 x 1024  103.9   34.4   24.5   20.4   22.7   28.4   23.5   29.8   25.1   28.2   33.9  s1
//    1024, 128 of 2048 x 1024  303.8   89.4   60.0   50.7   52.8   79.9   53.7   76.4   55.0   61.5   89.5  s1
//    8192, 128 of 2048 x 1024   1304  352.8  214.2  153.9  106.9  184.7   85.5  150.9   85.7   87.6  155.5  8/1
// The gradient (no kernel of few rows):
//   rows, matrices               2/1    2/2    2/4    2/8    4/1    4/2    6/1    6/2    8/1    8/2  rule
//      16, 4096 x 4096          20.1   15.3   12.7   12.7   22.9   17.0   27.6   19.5   30.5   21.2  2/4
//     512, 4096 x 4096          24.2   34.5   48.0   71.8   25.9   24.5   30.4   27.5   34.1   29.9  2/1
//     512, 8 of 4096 x 4096     47.4   50.6   61.9   95.8   33.0   43.2   33.8   36.7   34.8   37.1  4/1
//    2048, 8 of 4096 x 2048     66.9   79.3  103.7  160.9   51.4   60.1   35.1   51.5   38.9   62.7  6/1
//    1024, 128 of 2048 x 1024   49.7   61.2   80.9  127.6   50.6   61.8   52.3   66.4   56.1   71.1  2/1
// The choice is within 5% of the best of them but for 128 rows over 8 matrices (29.2
// for 24.7) and 8192 over 128 (91.6 for 85.5).  Sizes of the matrices on both sides of
// 64 MB, and matrices that the cache does not hold, were not compared.
struct BlockShape {
    int nt;
    int64_t splits;
    int waves;
};
static BlockShape block_shape(bool grad, bool direct, int64_t S, int64_t E, int64_t M, int64_t K) {
    const int64_t inner = grad ? M : K, outer = grad ? K : M, steps = blocks8(inner);
    BlockShape best{0, 1, 0};
    // (the copies of unaligned rows through registers take 16 codes of a row at least)
    if (inner < 16) return best;
    const int64_t live = S < E ? S : E;
    if (live < 1) return best;
    // an expert's last tile is half full on average
    auto tiles = [&](int64_t tt) {
        const int64_t half = S / tt + (live + 1) / 2;
        return E == 1 ? (S + tt - 1) / tt : half > live ? half : live;
    };
    const double bytes = (double)live * (double)M * (double)K, memory = bytes / 5.1e6;
    double least = 1e30;
    const double step_us[4] = {0.46, 0.6, 0.78, 0.95};
    for (int i = 0; i < 4; ++i) {
        const int64_t blocks = (outer + kTileRows - 1) / kTileRows * tiles(32 * (i + 1));
        const double step = bytes >= 64e6 && step_us[i] < 1.05 ? 1.05 : step_us[i];
        for (int64_t n = 1; n <= 16 && (n == 1 || steps / n >= 2); n *= 2) {
            const double rounds = (double)((blocks * n + 255) / 256), loop = rounds * (double)((steps + n - 1) / n) * step;
            double us = (loop > memory ? loop : memory) + 4.0 * rounds;
            if (n > 1) us += 4.0 + (double)(2 * n * S * outer) * sizeof(float) / 3.8e6;
            if (us < least) {
                least = us;
                best = {2 * (i + 1), n, 0};
            }
        }
    }
    // (the token tiles of a launch: 65535 at most)
    if (!grad && direct && S <= (int64_t)1 << 15) {
        const int64_t t16 = tiles(16), groups = (M + 31) / 32 * t16;
        const double read = (double)t16 * (double)M * (double)K / 1.1e7;
        const double us = 3.0 + (read > memory ? read : memory) * (t16 > live ? 1.2 : 1.0);
        if (us < least) best = {0, 1, (M + 15) / 16 * t16 <= 256 ? 8 : groups <= 512 ? 4 : groups < 2048 ? 2 : 1};
    }
    return best;
}

// (the workspace is asked for by sizes alone: enough for unaligned rows too)
static size_t block_scratch(bool grad, int64_t S, int64_t E, int64_t M, int64_t K) {
    const int64_t a = block_shape(grad, true, S, E, M, K).splits, b = block_shape(grad, false, S, E, M, K).splits;
    const int64_t n = a > b ? a : b;
    return n > 1 ? ((size_t)(n * S * (grad ? K : M)) * sizeof(float) + 255) & ~(size_t)255 : 0;
}
size_t block_product_scratch(int64_t S, int64_t E, int64_t M, int64_t K) { return block_scratch(false, S, E, M, K); }
size_t block_product_grad_scratch(int64_t S, int64_t E, int64_t M, int64_t K) { return block_scratch(true, S, E, M, K); }

template <typename O, bool GRAD>
static hipError_t block_launch(const BlockArgs& a, void* ws, hipStream_t s) {
    const int64_t inner = GRAD ? a.M : a.K, outer = GRAD ? a.K : a.M;
    const bool direct = inner % 16 == 0 && (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.codes % 16 == 0 && a.K % 16 == 0;
    const BlockShape shape = block_shape(GRAD, direct, a.S, a.E, a.M, a.K);
    hipError_t e = hipSuccess;
    if constexpr (!GRAD) {
#define KM_ST(WR, WK, R, NT)                                                                                            \
    do {                                                                                                                \
        constexpr int lds = BlockStream<WR, WK, R, NT>::BYTES;                                                          \
        if ((e = hipFuncSetAttribute((const void*)k_block_stream<O, WR, WK, R, NT>,                                     \
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds)) != hipSuccess)                   \
            return e;                                                                                                   \
        hipLaunchKernelGGL((k_block_stream<O, WR, WK, R, NT>),                                                          \
                           dim3((unsigned)((a.M + 16 * WR * R - 1) / (16 * WR * R)),                                    \
                                (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * NT)),                                 \
                           dim3(64 * WR * WK), lds, s, (const uint8_t*)a.x, a.x_scales, a.S, (const uint8_t*)a.codes,   \
                           a.scales, (int)a.E, a.M, a.K, a.offsets, a.order, a.top, (O*)a.out);                         \
        return hipGetLastError();                                                                                       \
    } while (0)
        switch (shape.waves) {
            case 8: KM_ST(1, 8, 1, 1);
            case 4: KM_ST(1, 4, 2, 1);
            case 2: KM_ST(2, 2, 2, 1);
            case 1: KM_ST(4, 1, 2, 1);
            default: break;
        }
#undef KM_ST
    }
    if (shape.nt == 0) {
        // (the grid's second axis holds 65535 token tiles)
        const int64_t all = segment_tiles(a.S, a.E, a.offsets, 16), most = 1 << 15;
        for (int64_t y0 = 0; y0 < all; y0 += most)
            hipLaunchKernelGGL((k_block_short<O, GRAD>),
                               dim3((unsigned)((outer + 15) / 16), (unsigned)(all - y0 < most ? all - y0 : most)), dim3(64), 0,
                               s, (const uint8_t*)a.x, a.x_scales, a.S, (const uint8_t*)a.codes, a.scales, (int)a.E, a.M,
                               a.K, a.offsets, a.order, a.top, y0, (O*)a.out);
        return hipGetLastError();
    }
    const int64_t steps = blocks8(inner), per = (steps + shape.splits - 1) / shape.splits;
    float* part = shape.splits > 1 ? (float*)ws : nullptr;
#define KM_GO2(NT, DIR)                                                                                                \
    do {                                                                                                               \
        constexpr int lds = BlockTile<NT>::BYTES;                                                                      \
        if ((e = hipFuncSetAttribute((const void*)k_block_tile<O, NT, GRAD, DIR>,                                      \
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds)) != hipSuccess)                  \
            return e;                                                                                                  \
        hipLaunchKernelGGL((k_block_tile<O, NT, GRAD, DIR>),                                                           \
                           dim3((unsigned)((outer + kTileRows - 1) / kTileRows),                                       \
                                (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * NT), (unsigned)shape.splits),        \
                           dim3(kTileThreads), lds, s, (const uint8_t*)a.x, a.x_scales, a.S, (const uint8_t*)a.codes,  \
                           a.scales, (int)a.E, a.M, a.K, a.offsets, a.order, a.top, per, (O*)a.out, part);             \
    } while (0)
#define KM_GO(NT)                      \
    do {                               \
        if (direct) KM_GO2(NT, true);  \
        else KM_GO2(NT, false);        \
    } while (0)
    if (shape.nt == 8) KM_GO(8);
    else if (shape.nt == 6) KM_GO(6);
    else if (shape.nt == 4) KM_GO(4);
    else KM_GO(2);
#undef KM_GO
#undef KM_GO2
    if ((e = hipGetLastError()) != hipSuccess || !part) return e;
    const int64_t n = a.S * outer;
    in_launches((n + 1023) / 1024, [&](int64_t b0, unsigned nb) {
        hipLaunchKernelGGL((k_block_join<O>), dim3(nb), dim3(256), 0, s, part, n, (int)shape.splits, (O*)a.out, b0);
    });
    return hipGetLastError();
}

hipError_t launch_block_product(DType ot, bool grad, const BlockArgs& a, void* ws, hipStream_t s) {
    if (a.S == 0) return hipSuccess;
#define KM_GO(O) return grad ? block_launch<O, true>(a, ws, s) : block_launch<O, false>(a, ws, s)
    if (ot == DType::F32) KM_GO(float);
    if (ot == DType::F16) KM_GO(_Float16);
    KM_GO(uint16_t);
#undef KM_GO
}

}  // namespace km

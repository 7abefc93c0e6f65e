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

// 16 bytes moved down by `by` (0 .. 15), zeros behind them.
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

// Many rows.  The same product on blocks of 64 WM rows of the matrix (GRAD: its
// columns) and 16 NT tokens; a wave has 64 of the rows and all of the tokens.
//
// A step takes 128 of the inner length.  The tokens' codes go to LDS by direct
// loads one step ahead, 16-byte chunks XOR-swizzled by the token, and are read by
// every wave; the matrix's come straight to operands (each wave has its own rows:
// nothing to share), also one step ahead.  GRAD wants columns of the matrix: a
// wave brings 128 rows by 64 columns to LDS and reads them transposed
// (ds_read_b64_tr_b8: a lane receives one column of eight rows).  The scales of 32
// steps lie in LDS.
//
// DIRECT: the rows of x (GRAD: of the matrix too) start at 16-byte boundaries;
// otherwise they are copied through registers, as is the last, partial step.
constexpr int kTileScales = 32;

template <bool V>
struct Tag {
    static constexpr bool value = V;
};
template <int V>
struct Int {
    static constexpr int value = V;
};

template <int WM, int NT, bool GRAD>
struct BlockTile {
    static constexpr int TT = 16 * NT, XROW = TT + 1;
    static constexpr int X = TT * kBlock8;             // a stage of tokens
    static constexpr int W = GRAD ? WM * 64 * kBlock8 : 0;  // and of the matrix
    static constexpr int SX = 2 * (X + W), SW = SX + kTileScales * XROW * 4;
    static constexpr int BYTES = SW + kTileScales * WM * 4;
};

// 16-byte chunk of row m (of 64 columns) that holds columns 16 c .. 16 c + 15: the
// 32 rows that a transposing read touches spread over all banks.
__device__ __forceinline__ int tile_chunk(int c, int m) { return c ^ ((m >> 2 & 1) ^ (m >> 4 & 3)); }

template <typename O, int WM, int NT, bool GRAD, bool DIRECT>
__global__ __launch_bounds__(64 * WM, 2) void k_block_tile(const uint8_t* __restrict__ x, const float* __restrict__ xs,
                                                           int64_t S, const uint8_t* __restrict__ codes,
                                                           const float* __restrict__ scales, int E, int64_t M,
                                                           int64_t K, const int32_t* __restrict__ offsets,
                                                           const int32_t* __restrict__ order, int64_t top,
                                                           O* __restrict__ out) {
    typedef BlockTile<WM, NT, GRAD> L;
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    constexpr int TT = L::TT, NTHR = 64 * WM, R = 4;
    constexpr int NX = TT * 8 / NTHR > 0 ? TT * 8 / NTHR : 1;  // a thread's chunks of a stage of tokens
    extern __shared__ __attribute__((aligned(16))) char s_mem[];
    float* s_x = (float*)(s_mem + L::SX);  // [32][XROW]
    float* s_w = (float*)(s_mem + L::SW);  // [32][WM]
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const Segment g = find_segment(offsets, S, E, TT, blockIdx.y);
    if (g.e < 0) return;
    const int64_t inner = GRAD ? M : K, outer = GRAD ? K : M, ib = blocks8(inner), kb = blocks8(K);
    const int64_t o0 = ((int64_t)blockIdx.x * WM + w) * 64;  // the wave's rows
    f32x4 acc[R][NT];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[a][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (g.e < E) {
        const int64_t whole = inner / kBlock8;
        const uint8_t* wm = codes + (int64_t)g.e * M * K;
        const float* ws = scales + (int64_t)g.e * blocks8(M) * kb;
        // a thread's chunks of tokens: 8 a token, chunk (lane & 7) ^ token at place lane & 7
        const uint8_t* xp[NX];
        const int xc = ((tid & 7) ^ (tid >> 3 & 7)) * 16;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int t = (i * NTHR + tid) >> 3;
            int64_t src = source_row(order, top, S, g.p0 + (t < g.n ? t : g.n - 1));
            xp[i] = x + (src < 0 ? 0 : src) * inner + xc;
        }
        // forward: rows a 16 + r of the wave's 64, from its first one
        const uint8_t* wb = wm + (GRAD ? 0 : (o0 < outer ? o0 : outer - 1) * K);
        uint32_t wo[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const int64_t left = outer - 1 - o0;  // (rows past the last one read it)
            wo[a] = (uint32_t)((a * 16 + r < left ? a * 16 + r : left < 0 ? 0 : left) * K) + q * 16;
        }
        auto xstage = [&](int b) { return s_mem + b * L::X; };
        auto wstage = [&](int b) { return s_mem + 2 * L::X + b * L::W + w * (64 * kBlock8); };
        // step st by direct loads: 1 KB an instruction
        auto fill = [&](int64_t st, int b) {
#pragma unroll
            for (int i = 0; i < NX; ++i)
                if (TT * 8 >= NTHR || tid < TT * 8) dma16_lane(xp[i] + st * kBlock8, xstage(b) + (i * NTHR + w * 64) * 16);
            if constexpr (GRAD) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // 16 rows of 64 columns; place lane & 3 of row m holds chunk tile_chunk(lane & 3, m)
                    const int m = i * 16 + (lane >> 2), c = tile_chunk(lane & 3, m);
                    const int64_t col = o0 + c * 16;
                    dma16_lane(wm + (st * kBlock8 + m) * K + (col < outer ? col : outer - 16), wstage(b) + i * 1024);
                }
            }
        };
        // the same through registers: loads now, stores later.  LAST: the partial step.
        auto copy_x = [&](int64_t st, u32x4 (&v)[NX], auto last_tag) {
            const int left = (int)(inner - st * kBlock8 < kBlock8 ? inner - st * kBlock8 : kBlock8);
#pragma unroll
            for (int i = 0; i < NX; ++i)
                if (TT * 8 >= NTHR || tid < TT * 8) {
                    if constexpr (decltype(last_tag)::value) v[i] = load16_end(xp[i] + st * kBlock8, left - xc, inner);
                    else v[i] = *(const u32x4_byte*)(xp[i] + st * kBlock8);
                }
        };
        auto keep_x = [&](int b, const u32x4 (&v)[NX]) {
#pragma unroll
            for (int i = 0; i < NX; ++i)
                if (TT * 8 >= NTHR || tid < TT * 8) *(u32x4*)(xstage(b) + (i * NTHR + tid) * 16) = v[i];
        };
        // (columns behind the row's end hold the next row's and give results that are not
        // stored; nothing behind the matrix is read)
        auto copy_w = [&](int64_t st, u32x4 (&v)[8], auto last_tag) {
            if constexpr (GRAD) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int m = i * 16 + (lane >> 2), c = tile_chunk(lane & 3, m);
                    const int64_t row = st * kBlock8 + m < M ? st * kBlock8 + m : M - 1, col = o0 + c * 16;
                    if constexpr (decltype(last_tag)::value) {
                        v[i] = load16_end(wm + row * K + (col < outer ? col : 0), (int)(outer - col < 16 ? outer - col : 16), K);
                    } else {
                        const int64_t at = row * K + (col < outer ? col : 0), over = at - (M * K - 16);
                        v[i] = *(const u32x4_byte*)(wm + (over > 0 ? M * K - 16 : at));
                        v[i] = move_down(v[i], over > 0 ? (int)over : 0);
                    }
                }
            }
        };
        auto keep_w = [&](int b, const u32x4 (&v)[8]) {
            if constexpr (GRAD) {
#pragma unroll
                for (int i = 0; i < 8; ++i) *(u32x4*)(wstage(b) + i * 1024 + lane * 16) = v[i];
            }
        };
        struct Part {
            i32x8 v[R];
        };
        auto fetch = [&](int64_t st, Part& p) {
            if constexpr (!GRAD) {
                const uint8_t* b = wb + st * kBlock8;
#pragma unroll
                for (int a = 0; a < R; ++a)
                    p.v[a] = join8(*(const u32x4_byte*)(b + wo[a]), *(const u32x4_byte*)(b + wo[a] + 64));
            }
        };
        auto fetch_end = [&](int64_t st, Part& p) {
            if constexpr (!GRAD) {
                const uint8_t* b = wb + st * kBlock8;
                const int left = (int)(inner - st * kBlock8) - q * 16;
#pragma unroll
                for (int a = 0; a < R; ++a)
                    p.v[a] = join8(load16_end(b + wo[a], left, K), load16_end(b + wo[a] + 64, left - 64, K));
            }
        };
        // the scales of the steps from st on
        auto fill_scales = [&](int64_t st) {
            for (int i = tid; i < TT * kTileScales; i += NTHR) {
                const int t = i / kTileScales, j = i % kTileScales;
                const int64_t src = source_row(order, top, S, g.p0 + (t < g.n ? t : g.n - 1));
                if (st + j < ib) s_x[j * L::XROW + t] = src < 0 ? 0.f : xs[src * ib + st + j];
            }
            for (int i = tid; i < WM * kTileScales; i += NTHR) {
                const int j = i / WM;
                const int64_t o = ((int64_t)blockIdx.x * WM + i % WM) * 64, ob = (o < outer ? o : outer - 1) / kBlock8;
                if (st + j < ib) s_w[i] = GRAD ? ws[(st + j) * kb + ob] : ws[ob * kb + st + j];
            }
        };
        auto multiply = [&](int64_t st, int b, const Part& p) {
            const int j = (int)(st % kTileScales);
            const float sw = s_w[j * WM + w];
            const char* xl = xstage(b);
            i32x8 av[R];
#pragma unroll
            for (int a = 0; a < R; ++a) {
                if constexpr (GRAD) {
                    // rows q 16 + (0 .. 15) and 64 more of column a 16 + r: a lane fetches 8 bytes of
                    // row r / 2 of eight, half r % 2 of the chunk
                    const char* wl = wstage(b);
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const int m = (f >> 1) * 64 + q * 16 + (f & 1) * 8 + (r >> 1);
                        const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                            (__attribute__((address_space(3))) i32x2*)(wl + m * 64 + tile_chunk(a, m) * 16 + (r & 1) * 8));
                        av[a][2 * f] = t[0];
                        av[a][2 * f + 1] = t[1];
                    }
                } else {
                    av[a] = p.v[a];
                }
            }
            // a result is scaled and added two instructions after its own was issued; the next
            // tokens are read while these are multiplied
            auto tokens = [&](int n) {
                const char* row = xl + (n * 16 + r) * kBlock8;
                return join8(*(const u32x4*)(row + ((q ^ (r & 7)) * 16)), *(const u32x4*)(row + (((q + 4) ^ (r & 7)) * 16)));
            };
            auto scale = [&](int n) { return sw * s_x[j * L::XROW + n * 16 + r]; };
            f32x4 d[3];
            i32x8 bv[2];
            float sc[2];
            bv[0] = tokens(0);
            sc[0] = scale(0);
#pragma unroll
            for (int i = 0; i < NT * R + 2; ++i) {
                const int n = i / R, a = i % R;
                if (a == 0 && n + 1 < NT) bv[(n + 1) & 1] = tokens(n + 1);
                if (a == 2 && n + 1 < NT) sc[(n + 1) & 1] = scale(n + 1);
                if (i < NT * R) d[i % 3] = mfma8(av[a], bv[n & 1], f32x4{0.f, 0.f, 0.f, 0.f});
                if (i >= 2) {
                    const int m = (i - 2) / R, c = (i - 2) % R;
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[c][m][e] = fmaf(sc[m & 1], d[(i - 2) % 3][e], acc[c][m][e]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        Part p[2];
        if (whole > 0) {
            fetch(0, p[0]);
            if constexpr (DIRECT) {
                fill(0, 0);
            } else {
                u32x4 xv[NX], wv[8];
                copy_x(0, xv, Tag<false>{});
                copy_w(0, wv, Tag<false>{});
                keep_x(0, xv);
                keep_w(0, wv);
            }
        }
        // The step of buffer b; the next one is on its way meanwhile (the last is fetched
        // twice rather than branched around: a branch here lets the compiler carry a step's
        // results over it and spill).
        auto step = [&](int64_t st, auto b_tag) {
            constexpr int b = decltype(b_tag)::value;
            if constexpr (DIRECT) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // this wave's direct loads, then everybody's
            __syncthreads();
            const int64_t next = st + 1 < whole ? st + 1 : st;
            u32x4 xv[NX], wv[8];
            fetch(next, p[b ^ 1]);
            if constexpr (DIRECT) {
                fill(next, b ^ 1);
            } else {
                copy_x(next, xv, Tag<false>{});
                copy_w(next, wv, Tag<false>{});
            }
            multiply(st, b, p[b]);
            if constexpr (!DIRECT) {
                keep_x(b ^ 1, xv);
                keep_w(b ^ 1, wv);
            }
        };
        auto refill = [&](int64_t st) {
            if (st % kTileScales == 0) {
                if (st) __syncthreads();  // the old ones have been read
                fill_scales(st);
            }
        };
        int64_t st = 0;
        for (; st + 1 < whole; st += 2) {
            refill(st);
            step(st, Int<0>{});
            step(st + 1, Int<1>{});
        }
        if (st < whole) {
            refill(st);
            step(st, Int<0>{});
        }
        if (whole < ib) {
            u32x4 xv[NX], wv[8];
            copy_x(whole, xv, Tag<true>{});
            copy_w(whole, wv, Tag<true>{});
            fetch_end(whole, p[0]);
            if constexpr (DIRECT) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // (the last fetch)
            __syncthreads();
            keep_x(0, xv);
            keep_w(0, wv);
            if (whole % kTileScales == 0) fill_scales(whole);
            __syncthreads();
            multiply(whole, 0, p[0]);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = n * 16 + r;
        if (t >= g.n) continue;
        // (a row of none: zeros, whatever row 0 held)
        const bool none = order && g.e < E && source_row(order, top, S, g.p0 + t) < 0;
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const int64_t o = o0 + a * 16 + q * 4;
            if (o < outer)
                store_results<O>(out + (g.p0 + t) * outer + o, outer - o, none ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[a][n]);
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
#define KM_GO2(WM, NT, DIR)                                                                                            \
    do {                                                                                                               \
        constexpr int lds = BlockTile<WM, NT, GRAD>::BYTES;                                                            \
        if (lds > 64 * 1024 &&                                                                                         \
            (e = hipFuncSetAttribute((const void*)k_block_tile<O, WM, NT, GRAD, DIR>,                                  \
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds)) != hipSuccess)                  \
            return e;                                                                                                  \
        hipLaunchKernelGGL((k_block_tile<O, WM, NT, GRAD, DIR>),                                                       \
                           dim3((unsigned)((outer + 64 * WM - 1) / (64 * WM)),                                         \
                                (unsigned)segment_tiles(a.S, a.E, a.offsets, 16 * NT)),                                \
                           dim3(64 * WM), lds, s, KM_ARGS);                                                            \
    } while (0)
#define KM_GO(WM, NT)                      \
    do {                                   \
        if (direct) KM_GO2(WM, NT, true);  \
        else KM_GO2(WM, NT, false);        \
    } while (0)
    if (a.S >= 32 * a.E) {
        KM_GO(4, 8);
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

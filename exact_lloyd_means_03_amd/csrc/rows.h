// Access to rows of d elements in pieces of 16 bytes, shared by the kernels
// that gather, scatter and combine whole rows (rows.hip, lookup_grad.hip).
//
// A row is cut into row_chunks(d) chunks of RowVec<T>::N elements.  Where d
// is no multiple of N the last chunk is moved back to end with the row: it
// overlaps the one before it, both hold the same values there, and no lane
// runs an element loop (rows shorter than one chunk do).  Rows start at any
// element boundary: the vectors are declared with the element's alignment,
// which gfx950's global loads and stores accept.
#pragma once

#include "common.h"

namespace km {

template <typename T>
struct RowVec {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
    typedef V VU __attribute__((aligned(sizeof(T))));
};

inline int row_chunks(int64_t d, int es) { return (int)((d * es + 15) / 16); }

// First element of chunk c, and the elements a chunk holds.
template <typename T>
__device__ __forceinline__ int chunk_at(int c, int d) {
    constexpr int N = RowVec<T>::N;
    return (c + 1) * N <= d ? c * N : (d > N ? d - N : 0);
}

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float elem_f32(uint16_t v) { return bf16_to_f32(v); }

template <typename T>
__device__ __forceinline__ T elem_from(float v);
template <>
__device__ __forceinline__ float elem_from<float>(float v) { return v; }
template <>
__device__ __forceinline__ _Float16 elem_from<_Float16>(float v) {
    // the float32 value is formed first: folded into a mixed-precision multiply
    // it would be rounded from the exact product, unlike the other types
    asm("" : "+v"(v));
    return (_Float16)v;
}
template <>
__device__ __forceinline__ uint16_t elem_from<uint16_t>(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
}

// The chunk's bits at p (d elements in the row; shorter rows are zero-filled).
template <typename T>
__device__ __forceinline__ typename RowVec<T>::V load_raw(const T* __restrict__ p, int d) {
    using R = RowVec<T>;
    if (d >= R::N) return *(const typename R::VU*)p;
    typename R::V v{};
    for (int i = 0; i < d; ++i) v[i] = p[i];
    return v;
}

// STREAM: a non-temporal store, for results of half the memory-side cache's
// 256 MB or more: with the inputs beside them they would not all be found there
// by whoever reads them next; kept out of it, they neither evict the operator's
// inputs nor have to be written back while the next launch reads (lookup of
// 49999 rows of 8 KB: 112 -> 82 us; dispatch and combine of 98526 rows of 4 KB:
// 74 + 128 -> 85 + 87 us).
inline bool stream_out(int64_t bytes) { return bytes >= ((int64_t)128 << 20); }
template <typename T, bool STREAM = false>
__device__ __forceinline__ void store_raw(T* __restrict__ p, int d, typename RowVec<T>::V v) {
    using R = RowVec<T>;
    if (d >= R::N) {
        if constexpr (STREAM) __builtin_nontemporal_store(v, (typename R::VU*)p);
        else *(typename R::VU*)p = v;
    } else {
        for (int i = 0; i < d; ++i) p[i] = v[i];
    }
}

// N float32 values (of which d are in the row, if it is shorter) as T.
template <typename T, int N, bool STREAM = false>
__device__ __forceinline__ void store_f32(T* __restrict__ p, int d, const float (&a)[N]) {
    constexpr int VN = RowVec<T>::N;  // N is VN, or 2 VN: float32 results of a 16-bit chunk
    static_assert(N == VN || N == 2 * VN, "one vector or two");
    typename RowVec<T>::V v;
#pragma unroll
    for (int i = 0; i < VN; ++i) v[i] = elem_from<T>(a[i]);
    store_raw<T, STREAM>(p, d, v);
    if constexpr (N > VN) {
#pragma unroll
        for (int i = 0; i < VN; ++i) v[i] = elem_from<T>(a[VN + i]);
        // d >= N or the row ends in one of the two vectors
        if (d > VN) store_raw<T, STREAM>(p + VN, d - VN, v);
    }
}

// A launch has fewer than 2^32 threads (hipLaunchKernel's limit in a dimension
// of the grid): more blocks than kLaunchBlocks of 256 threads are launched in
// parts, launch(first block, blocks); blocks of up to 64 `waves` threads where
// waves is above 4.
constexpr int64_t kLaunchBlocks = (int64_t)1 << 22;
template <typename F>
inline void in_launches(int64_t blocks, F launch, int waves = 4) {
    const int64_t most = waves > 4 ? kLaunchBlocks * 4 / waves : kLaunchBlocks;
    for (int64_t b0 = 0; b0 < blocks; b0 += most) launch(b0, (unsigned)(blocks - b0 < most ? blocks - b0 : most));
}

// Items (row, chunk) of a launch are numbered row-major; block b of threads
// starts at item b * per_block.  item_at splits the item `off` places after
// the block's first one without a 64-bit division per thread.
struct ItemBase {
    int64_t row;
    uint32_t chunk;
};
__device__ __forceinline__ ItemBase item_base(int64_t block0, int64_t per_block, uint32_t C) {
    const uint64_t first = (uint64_t)(block0 + blockIdx.x) * (uint64_t)per_block;
    const uint64_t r = first / C;
    return {(int64_t)r, (uint32_t)(first - r * C)};
}
__device__ __forceinline__ void item_at(const ItemBase& base, uint32_t off, uint32_t C, int64_t* row, int* chunk) {
    const uint32_t x = base.chunk + off, q = x / C;
    *row = base.row + q;
    *chunk = (int)(x - q * C);
}

}  // namespace km

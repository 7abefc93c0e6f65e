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

template <typename T>
__device__ __forceinline__ void store_raw(T* __restrict__ p, int d, typename RowVec<T>::V v) {
    using R = RowVec<T>;
    if (d >= R::N) {
        *(typename R::VU*)p = v;
    } else {
        for (int i = 0; i < d; ++i) p[i] = v[i];
    }
}

// The first n (<= N) elements from float32.
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* __restrict__ p, int d, const float (&a)[N]) {
    if constexpr (N == RowVec<T>::N) {
        typename RowVec<T>::V v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = elem_from<T>(a[i]);
        store_raw<T>(p, d, v);
    } else {
        // float32 results of a 16-bit chunk: two vectors
        static_assert(N == 2 * RowVec<T>::N, "a 16-bit chunk holds twice a float32 chunk");
        if (d >= N) {
            typename RowVec<T>::V lo, hi;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                lo[i] = elem_from<T>(a[i]);
                hi[i] = elem_from<T>(a[N / 2 + i]);
            }
            *(typename RowVec<T>::VU*)p = lo;
            *(typename RowVec<T>::VU*)(p + N / 2) = hi;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < d) p[i] = elem_from<T>(a[i]);
        }
    }
}

// Items (row, chunk) of a launch are numbered row-major; block b of threads
// starts at item b * per_block.  ItemAt splits the item `off` places after
// the block's first one without a 64-bit division per thread.
struct ItemBase {
    int64_t row;
    uint32_t chunk;
};
__device__ __forceinline__ ItemBase item_base(int64_t per_block, uint32_t C) {
    const uint64_t first = (uint64_t)blockIdx.x * (uint64_t)per_block;
    const uint64_t r = first / C;
    return {(int64_t)r, (uint32_t)(first - r * C)};
}
__device__ __forceinline__ void item_at(const ItemBase& base, uint32_t off, uint32_t C, int64_t* row, int* chunk) {
    const uint32_t x = base.chunk + off, q = x / C;
    *row = base.row + q;
    *chunk = (int)(x - q * C);
}

}  // namespace km

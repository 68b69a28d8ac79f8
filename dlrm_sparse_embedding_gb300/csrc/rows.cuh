// Rows of a matrix as the dense side's kernels read and write them (sm_103a).
#pragma once

#include <type_traits>

#include "dense_internal.cuh"

namespace emb {

// V consecutive elements: 8 (moved 16 bytes at a time) where everything is
// aligned for it, else 2 where everything is for that, else 1.  They are kept as they
// are in memory until they are used: a load in flight costs no more registers than its
// bytes.  Rows are read and written once, so vectors pass as streams, which leave L2
// first (gradients and weighted sum of 32768 x 4 x 2048 together 299 us without, 273
// with).
template <int V, class T>
struct WordOf { using type = uint4; };
template <class T>
struct WordOf<4, T> { using type = typename std::conditional<sizeof(T) == 2, uint2, uint4>::type; };
template <class T>
struct WordOf<2, T> { using type = typename std::conditional<sizeof(T) == 2, uint32_t, uint2>::type; };
template <class T>
struct WordOf<1, T> { using type = T; };

template <int V, class T>
struct Raw {
    using Word = typename WordOf<V, T>::type;
    static constexpr int kWords = V * sizeof(T) / sizeof(Word);
    Word w[kWords];

    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (V > 1) w[i] = __ldcs(reinterpret_cast<const Word*>(p) + i);
            else w[i] = p[i];
        }
    }
    // what is read again soon
    __device__ __forceinline__ void load_again(const T* p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const Word*>(p) + i);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = Word{};
    }
    // from shared memory
    __device__ __forceinline__ void load_shared(const T* p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const Word*>(p)[i];
    }
    __device__ __forceinline__ float operator[](int i) const { return to_float<T>(reinterpret_cast<const T*>(w)[i]); }
};

template <int V, class T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V])
{
    using Word = typename Raw<V, T>::Word;
    Raw<V, T> r;
#pragma unroll
    for (int i = 0; i < V; ++i) reinterpret_cast<T*>(r.w)[i] = from_float<T>(v[i]);
#pragma unroll
    for (int i = 0; i < Raw<V, T>::kWords; ++i) {
        if constexpr (V > 1) __stcs(reinterpret_cast<Word*>(p) + i, r.w[i]);
        else p[i] = r.w[i];
    }
}

// How many elements of such rows can be moved at a time.
inline int vector_of(const void* p, int dtype, int64_t stride, int64_t width)
{
    const int64_t bytes = dtype_bytes(dtype);
    if (aligned_to(p, 16) && stride * bytes % 16 == 0 && width % 8 == 0) return 8;
    return aligned_to(p, 2 * bytes) && stride % 2 == 0 && width % 2 == 0 ? 2 : 1;
}

inline bool rows_valid(const void* p, int dtype, int64_t stride, int64_t width, int64_t n)
{
    return dtype_valid(dtype) && stride >= width && aligned_to(p, dtype_bytes(dtype)) && (p || n == 0);
}

template <class F>
int with_type(int dtype, F f)
{
    if (dtype == EMB_F32) return f(float());
    if (dtype == EMB_F16) return f(__half());
    return f(__nv_bfloat16());
}

}  // namespace emb

// The orthogonalisation's two ways through its steps (sm_103a).
#pragma once

#include <cmath>

#include "product_core.cuh"

namespace emb {

// A number is held as fp16 h plus fp16 l / kLowScale: l is h's rounding error,
// at most 2^-11 |h|, scaled up so that it is not lost where h is subnormal.
constexpr float kLowScale = 2048.f;

// Longest short side that orthogonal_short.cu takes: one operand of a CTA.
constexpr int kShort = core::kRows;

// X in the workspace, and what is done with it.
struct StepsArgs {
    __half *x[2], *x_low[2];    // [batch][rows][ld]; x[0] (and x_low[0], if low_in) holds 2^e G
    bool low_in;
    const float* scale;         // of each matrix: what takes 2^e G to 2^lift X0
    const int* lift;
    int64_t batch, rows, cols, ld;
    int steps;
    float a, b, c;
    __nv_bfloat16* out;         // [batch][rows][cols]
    __half *w, *w_low;          // short sides: [batch][kShort][kShort]
};

int run_short(const StepsArgs& p, cudaStream_t st);

// Where |G| is far below eps, X is far below 1 and would fall through fp16's 2^-24 (its
// low part's 2^-35).  It is held times 2^lift, which starts at what brings X0's norm to
// [0.5, 1) and goes down as fast as X can grow while it is small, by |a| a step: X in
// memory stays at most about 1, and the last one is X itself.  (256 x 512 of norm 1e-15
// at eps 1e-7: 9% off without, as much as any other with.)
struct Lift {
    const int* first;    // of each matrix
    float down;          // log2 of a step's growth
    int steps;
    __device__ int at(int64_t matrix, int step) const
    {
        return step < steps ? max(0, first[matrix] - (int)ceilf(step * down)) : 0;
    }
    // what X X^T as it is in memory is to be multiplied by, and X from one step to another
    __device__ float of_square(int64_t matrix, int step) const { return ldexpf(1.f, -2 * at(matrix, step)); }
    __device__ float between(int64_t matrix, int step, int next) const { return ldexpf(1.f, at(matrix, next) - at(matrix, step)); }
};
inline Lift lift_of(const int* first, float a, int steps)
{
    const float down = std::log2(std::fabs(a));
    return Lift{first, down > 0.f ? down : 0.f, steps};
}

// Two fp32 products and sums at once, each rounded once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight fp16 numbers as four pairs.
__device__ __forceinline__ void unpack8(const uint4& p, float2 (&v)[4])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float2 (&v)[4])
{
    return make_uint4(core::pack2<T>(v[0].x, v[0].y), core::pack2<T>(v[1].x, v[1].y), core::pack2<T>(v[2].x, v[2].y), core::pack2<T>(v[3].x, v[3].y));
}

// h + l / kLowScale
__device__ __forceinline__ void join8(const uint4& high, const uint4& low, float2 (&v)[4])
{
    float2 l[4];
    unpack8(high, v);
    unpack8(low, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(both(1.f / kLowScale), l[i], v[i]);
}

// v as two fp16 numbers each.
__device__ __forceinline__ void split8(const float2 (&v)[4], uint4& high, uint4& low)
{
    high = pack8<__half>(v);
    float2 h[4], l[4];
    unpack8(high, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = mul2(sub2(v[i], h[i]), both(kLowScale));
    low = pack8<__half>(l);
}

}  // namespace emb

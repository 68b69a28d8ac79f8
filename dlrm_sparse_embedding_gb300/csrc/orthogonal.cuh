// The orthogonalisation's two ways through its steps (sm_103a).
#pragma once

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
    const float* scale;         // of each matrix: what takes 2^e G to X0
    int64_t batch, rows, cols, ld;
    int steps;
    float a, b, c;
    __nv_bfloat16* out;         // [batch][rows][cols]
    __half *w, *w_low;          // short sides: [batch][kShort][kShort]
};

int run_short(const StepsArgs& p, cudaStream_t st);

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

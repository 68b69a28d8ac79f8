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

__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

// v as two fp16 numbers each, two at a time.
__device__ __forceinline__ void split8(const float (&v)[8], uint4& high, uint4& low)
{
    high = core::pack8<__half>(v);
    const uint32_t h[4] = {high.x, high.y, high.z, high.w};
    uint32_t l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 off = sub2(make_float2(v[2 * i], v[2 * i + 1]), __half22float2(*reinterpret_cast<const __half2*>(&h[i])));
        const float2 up = mul2(off, make_float2(kLowScale, kLowScale));
        l[i] = core::pack2<__half>(up.x, up.y);
    }
    low = make_uint4(l[0], l[1], l[2], l[3]);
}

}  // namespace emb

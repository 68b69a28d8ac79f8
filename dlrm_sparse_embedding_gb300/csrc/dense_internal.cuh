// Internal declarations of the expert and orthogonalisation calls (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "emb.h"
#include "launch.cuh"

namespace emb {

constexpr int kMaxExperts = 1024;
constexpr int kMaxExpertsPerToken = 64;

// The device's sticky status word (ERRBIT_* of emb_internal.cuh), or null when
// it cannot be had; experts.cu.
int* dense_status_word();

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t dtype_bytes(int dtype) { return dtype == EMB_F32 ? 4 : 2; }
inline bool dtype_valid(int dtype) { return dtype == EMB_F32 || dtype == EMB_F16 || dtype == EMB_BF16; }

// Whether the host can use the plan: sizes within the limits, arrays aligned.
bool expert_plan_valid(const emb_expert_plan* plan);

template <class T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Offset e of a plan, clamped into [0, P]: a plan that is not one never sends
// a kernel outside its arrays.
__device__ __forceinline__ int plan_offset(const int32_t* offsets, int e, int P)
{
    const int v = offsets[e];
    return v < 0 ? 0 : (v > P ? P : v);
}

}  // namespace emb

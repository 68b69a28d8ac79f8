// The experts' forward product for a handful of rows (single samples being served).
//
// One row uses each of its expert's weights once, so the product is bound by
// reading them: at 128 x 128 a tile, a row of 1024 outputs would keep 8 of the
// 152 SMs busy.  Here a warp has one output of one row, in fp32, and reads the
// weights 16 bytes a lane, whole sectors at a time.  Rows that share an expert
// read its weights again, from L2.  Weights from memory, rows of different experts
// (of one): 3328 x 1024 takes 4.4 us for one row and 8.7 (6.4) for four, in tiles
// 12.9 and 19.2 (12.9); 1024 x 4096 3.4 and 10.8 (8.5), in tiles 7.8 and 12.2 (7.7).
// From five rows on, those that share experts are faster in tiles (1024 x 4096:
// 8.0 us for 10.3; of different experts 15.3 for 12.8), so kFewRows ends it there.
// (A gradient's rows have the weights' long side as their sum's other one and fill the
// GPU with tiles: 8.7 us against 9.3 for two rows at 3328 x 1024 when it was written
// this way.)
#include "products.cuh"

namespace emb {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// The expert of row p: how many groups end at or before it; >= experts for a row without one.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int experts, int p)
{
    int n = 0;
    for (int base = 0; base < experts; base += kThreads) {
        const int e = base + threadIdx.x;
        n += __syncthreads_count(e < experts && offsets[e + 1] <= p);
    }
    return n;
}

template <class T>
__device__ __forceinline__ void unpack(const uint4& r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float<T>(reinterpret_cast<const T*>(&r)[i]);
}

// y[p][n] = <weight[e][n], rows[p]>
template <class T>
__global__ void __launch_bounds__(kThreads) few_forward(const T* __restrict__ rows, int64_t rows_stride, const T* __restrict__ weight,
                                                        int64_t in_width, int64_t out_width, const int32_t* __restrict__ offsets,
                                                        int experts, T* __restrict__ y)
{
    let_next_begin();
    wait_for_earlier();
    const int p = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int e = expert_of(offsets, experts, p);
    if (n >= out_width) return;
    float sum = 0.f;
    if (e < experts) {
        const uint4* const w = reinterpret_cast<const uint4*>(weight + (e * out_width + n) * in_width);
        const uint4* const x = reinterpret_cast<const uint4*>(rows + p * rows_stride);
        const int pieces = (int)(in_width / 8);
        constexpr int kAhead = 8;
        for (int c0 = lane; c0 < pieces; c0 += 32 * kAhead) {
            uint4 wv[kAhead], xv[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (c0 + 32 * i < pieces) wv[i] = __ldg(w + c0 + 32 * i), xv[i] = __ldg(x + c0 + 32 * i);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (c0 + 32 * i < pieces) {
                    float a[8], b[8];
                    unpack<T>(wv[i], a);
                    unpack<T>(xv[i], b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = __fmaf_rn(a[j], b[j], sum);
                }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (lane == 0) y[p * out_width + n] = from_float<T>(sum);
}

}  // namespace

int launch_few_rows(const ProductArgs& p, cudaStream_t st)
{
    const auto go = [&](auto t) {
        using T = decltype(t);
        const dim3 grid((unsigned)((p.n + kWarps - 1) / kWarps), (unsigned)p.m);
        return launch_next(few_forward<T>, grid, kThreads, 0, st, 1, (const T*)p.a, p.lda, (const T*)p.b, p.k, p.n, p.offsets, p.experts, (T*)p.d);
    };
    return p.dtype == EMB_F16 ? go(__half()) : go(__nv_bfloat16());
}

}  // namespace emb

// Matrix products of the expert layer and of the orthogonalisation.
#include "products.cuh"

namespace emb {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <class T>
__device__ __forceinline__ float element(const void* p, int64_t ld, bool mn, int64_t r, int64_t k)
{
    return to_float<T>(static_cast<const T*>(p)[mn ? k * ld + r : r * ld + k]);
}

// One 64 x 64 tile of one problem a block; a thread has 4 x 4 of it.
template <class T>
__global__ void __launch_bounds__(kThreads) product_tiles(ProductArgs p, int experts)
{
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    const int t = threadIdx.x, tm = t / 16, tn = t % 16;
    int64_t m0 = (int64_t)blockIdx.y * kTile, m_end = p.m, k0 = 0, k_end = p.k;
    const int64_t n0 = (int64_t)blockIdx.x * kTile;
    int problem = blockIdx.z;
    const int P = (int)(p.k_grouped ? p.k : p.m);
    bool tail = false;
    if (p.m_grouped) {   // blockIdx.y counts the groups' tiles one after another; the rows after them are zeroed
        int64_t left = blockIdx.y;
        int first = 0;
        for (problem = 0; problem <= experts; ++problem) {
            const int lo = max(first, plan_offset(p.offsets, problem, P));
            const int hi = problem < experts ? max(lo, plan_offset(p.offsets, problem + 1, P)) : P;
            const int64_t tiles = (hi - lo + kTile - 1) / kTile;
            if (left < tiles) {
                m0 = lo + left * kTile;
                m_end = hi;
                break;
            }
            left -= tiles;
            first = lo;
        }
        if (problem > experts) return;
        tail = problem == experts;
    }
    if (p.k_grouped) {
        k0 = plan_offset(p.offsets, problem, P);
        k_end = max((int64_t)k0, (int64_t)plan_offset(p.offsets, problem + 1, P));
    }
    const T* const a = static_cast<const T*>(p.a) + (p.m_grouped || p.k_grouped ? 0 : problem * p.batch_a);
    const T* const b = static_cast<const T*>(p.b) + (p.k_grouped || tail ? 0 : problem * p.batch_b);
    float acc[4][4] = {};
    if (!tail)
        for (int64_t k = k0; k < k_end; k += kStep) {
            for (int i = t; i < kTile * kStep; i += kThreads) {
                const int r = p.a_mn ? i % kTile : i / kStep, c = p.a_mn ? i / kTile : i % kStep;
                as[c][r] = m0 + r < m_end && k + c < k_end ? element<T>(a, p.lda, p.a_mn, m0 + r, k + c) : 0.f;
                const int rb = p.b_mn ? i % kTile : i / kStep, cb = p.b_mn ? i / kTile : i % kStep;
                bs[cb][rb] = n0 + rb < p.n && k + cb < k_end ? element<T>(b, p.ldb, p.b_mn, n0 + rb, k + cb) : 0.f;
            }
            __syncthreads();
            for (int c = 0; c < kStep; ++c)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(as[c][tm * 4 + i], bs[c][tn * 4 + j], acc[i][j]);
            __syncthreads();
        }
    float s = 1.f;
    if (p.scale) {
        s = p.scale[problem];
        if (p.scale_power == 2) s *= s;
    }
    const int64_t at_c = p.m_grouped ? 0 : problem * p.batch_c, at_d = p.m_grouped ? 0 : problem * p.batch_d;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + tm * 4 + i, n = n0 + tn * 4 + j;
            if (m >= m_end || n >= p.n) continue;
            float v = p.alpha * acc[i][j];
            if (p.c) {
                float c = __half2float(static_cast<const __half*>(p.c)[at_c + m * p.ldc + n]);
                if (p.c_low) c = __fmaf_rn(1.f / kLowScale, __half2float(static_cast<const __half*>(p.c_low)[at_c + m * p.ldc + n]), c);
                v = __fmaf_rn(p.beta, c, v);
            }
            v *= s;
            if (m == n) v += p.diagonal;
            const int64_t at = at_d + m * p.ldd + n;
            if (p.d_dtype == EMB_BF16) {
                static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16_rn(v);
            } else {
                const __half h = __float2half_rn(v);
                static_cast<__half*>(p.d)[at] = h;
                if (p.d_low) static_cast<__half*>(p.d_low)[at] = __float2half_rn(kLowScale * (v - __half2float(h)));
            }
        }
}

}  // namespace

int launch_product(const ProductArgs& p, cudaStream_t st)
{
    const int64_t tm = (p.m + kTile - 1) / kTile, tn = (p.n + kTile - 1) / kTile;
    const dim3 grid((unsigned)tn, (unsigned)(p.m_grouped ? tm + p.batch + 1 : tm), (unsigned)(p.m_grouped ? 1 : p.batch));
    if (p.dtype == EMB_F16)
        product_tiles<__half><<<grid, kThreads, 0, st>>>(p, (int)p.batch);
    else
        product_tiles<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p, (int)p.batch);
    return cudaGetLastError() == cudaSuccess ? EMB_OK : EMB_ERR_CUDA;
}

}  // namespace emb

using namespace emb;

namespace {

bool linear_valid(const emb_expert_plan* plan, int64_t in_width, int64_t out_width, int dtype)
{
    return expert_plan_valid(plan) && (dtype == EMB_F16 || dtype == EMB_BF16) && in_width >= 8 && out_width >= 8 &&
           in_width % 8 == 0 && out_width % 8 == 0 && in_width <= (1 << 24) && out_width <= (1 << 24);
}

bool array_valid(const void* p, int64_t stride, int64_t width, int64_t n)
{
    return (p || n == 0) && aligned_to(p, 16) && stride >= width && stride % 8 == 0;
}

}  // namespace

extern "C" int emb_expert_linear(const emb_expert_plan* plan, const void* rows, int64_t rows_stride, const void* weight,
                                 int64_t in_width, int64_t out_width, int32_t dtype, void* y, void* stream)
{
    if (!linear_valid(plan, in_width, out_width, dtype) || !array_valid(rows, rows_stride, in_width, plan->tokens) ||
        !array_valid(weight, in_width, in_width, 1) || !array_valid(y, out_width, out_width, plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    ProductArgs p;
    p.dtype = p.d_dtype = dtype;
    p.a = rows, p.lda = rows_stride;
    p.b = weight, p.ldb = in_width, p.batch_b = in_width * out_width;
    p.m = plan->tokens * plan->k, p.n = out_width, p.k = in_width;
    p.offsets = plan->offsets, p.m_grouped = true, p.batch = plan->experts;
    p.d = y, p.ldd = out_width;
    return launch_product(p, static_cast<cudaStream_t>(stream));
}

extern "C" int emb_expert_linear_grad_rows(const emb_expert_plan* plan, const void* grad_y, int64_t grad_stride, const void* weight,
                                           int64_t in_width, int64_t out_width, int32_t dtype, void* grad_rows, void* stream)
{
    if (!linear_valid(plan, in_width, out_width, dtype) || !array_valid(grad_y, grad_stride, out_width, plan->tokens) ||
        !array_valid(weight, in_width, in_width, 1) || !array_valid(grad_rows, in_width, in_width, plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    ProductArgs p;
    p.dtype = p.d_dtype = dtype;
    p.a = grad_y, p.lda = grad_stride;
    p.b = weight, p.ldb = in_width, p.b_mn = true, p.batch_b = in_width * out_width;
    p.m = plan->tokens * plan->k, p.n = in_width, p.k = out_width;
    p.offsets = plan->offsets, p.m_grouped = true, p.batch = plan->experts;
    p.d = grad_rows, p.ldd = in_width;
    return launch_product(p, static_cast<cudaStream_t>(stream));
}

extern "C" int emb_expert_linear_grad_weight(const emb_expert_plan* plan, const void* grad_y, int64_t grad_stride,
                                             const void* rows, int64_t rows_stride, int64_t in_width, int64_t out_width,
                                             int32_t dtype, void* grad_weight, void* stream)
{
    if (!linear_valid(plan, in_width, out_width, dtype) || !array_valid(grad_y, grad_stride, out_width, plan->tokens) ||
        !array_valid(rows, rows_stride, in_width, plan->tokens) || !array_valid(grad_weight, in_width, in_width, 1))
        return EMB_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (plan->tokens == 0)
        return cudaMemsetAsync(grad_weight, 0, (size_t)plan->experts * in_width * out_width * 2, st) == cudaSuccess ? EMB_OK : EMB_ERR_CUDA;
    ProductArgs p;
    p.dtype = p.d_dtype = dtype;
    p.a = grad_y, p.lda = grad_stride, p.a_mn = true;
    p.b = rows, p.ldb = rows_stride, p.b_mn = true;
    p.m = out_width, p.n = in_width, p.k = plan->tokens * plan->k;
    p.offsets = plan->offsets, p.k_grouped = true, p.batch = plan->experts;
    p.d = grad_weight, p.ldd = in_width, p.batch_d = in_width * out_width;
    return launch_product(p, st);
}

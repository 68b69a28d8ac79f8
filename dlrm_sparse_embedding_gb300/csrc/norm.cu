// Layer norm: the calls, how rows are laid on the grid, and the sum of the blocks' parts
// of the parameters' gradients.
#include "norm.cuh"

#include <algorithm>
#include <cmath>

namespace emb {
namespace norm {
namespace {

constexpr int kSms = 152;
constexpr int64_t kMaxWidth = 1 << 24;

// Threads a row and elements a thread (the same for a gradient of any alignment).  Up to a warp the threads are a power of two and
// a warp takes several rows; beyond, whole warps and one row a block.  The grid is what
// the GPU holds at once: a block goes through its rows with the next ones on their way.
Shape shape_of(int64_t rows, int64_t width, bool grad, bool vectors)
{
    Shape s = {};
    // of few rows, all on their way at once, more threads have less to do one after another (1 x 3328: 4.5 us for 6.1)
    const int most = grad || !vectors || (rows <= kSms && width <= kMaxThreads * kFew) ? kFew : kMany;
    s.chunks = 1;
    if (width > kMaxThreads * most) {
        s.kind = kWideRows;
        s.tx = kWideThreads, s.ty = 1;
        s.blocks = (int)std::min<int64_t>(rows, 2 * kSms);
        const int64_t columns = (width + 127) / 128;   // blocks of the column sums across a row, of vectors of 4
        s.chunks = (int)std::max<int64_t>(1, std::min((rows + 4 * kColumnRows - 1) / (4 * kColumnRows), 8 * kSms / columns));
        return s;
    }
    s.kind = width <= 32 * most ? kWarpRows : kBlockRows;
    s.per_thread = width <= 32 * kFew ? kFew : most;
    const int threads = (int)((width + s.per_thread - 1) / s.per_thread);
    if (s.kind == kWarpRows) {
        for (s.tx = 1; s.tx < threads;) s.tx *= 2;
        s.ty = kThreads / s.tx;
    } else {
        s.tx = (threads + 31) / 32 * 32;
        // A gradient's short rows share a block by as many as leave the SM as many rows as ones alone would: 20000 x 1536
        // bf16 48.5 us with five, 52 with two; of more than four warps a row alone (16384 x 3328 87 us, with two 91).
        const int held = 65536 / (registers(s.per_thread, grad, vectors) * s.tx);
        s.ty = !grad || s.tx > 128 ? 1 : held <= kMaxSubs ? held : held / 2;
    }
    s.per_sm = std::max(1, std::min(8, 65536 / (registers(s.per_thread, grad, vectors) * s.tx * s.ty)));
    if (s.kind == kBlockRows) s.per_sm = std::max(1, std::min(s.per_sm, kSharedBytes / (int)(3 * width * s.ty * (grad ? 8 : 4) + kOwnBytes)));
    s.blocks = (int)std::min<int64_t>((rows + s.ty - 1) / s.ty, (int64_t)kSms * s.per_sm);
    return s;
}

// Parts that the parameters' gradients come in.
int64_t parts_of(const Shape& s) { return s.kind == kWideRows ? s.chunks : s.blocks; }

size_t stats_bytes(const Shape& s, int64_t rows) { return s.kind == kWideRows ? (size_t)rows * sizeof(float4) : 0; }

bool sizes_valid(int64_t rows, int64_t width) { return rows >= 0 && width >= 1 && width <= kMaxWidth && rows <= (int64_t(1) << 40); }

// out[column] = the sum of the parts, 32 groups of them side by side.
constexpr int kGroups = 32;
__global__ void __launch_bounds__(32 * kGroups) sum_parts(const float* __restrict__ partial, int parts, int width, int dtype, void* dw, void* db)
{
    __shared__ float sums[kGroups][33];
    let_next_begin();
    wait_for_earlier();
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x, stride = 2 * (int64_t)width;   // dw's columns, then db's
    float s = 0.f;
    if (c < stride) {
#pragma unroll 8
        for (int p = threadIdx.y; p < parts; p += kGroups) s += partial[p * stride + c];
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = sums[threadIdx.x][threadIdx.y];   // a warp adds up one column's groups
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const int64_t mine = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && mine < stride) {
        void* const to = mine < width ? dw : db;
        const int64_t i = mine < width ? mine : mine - width;
        if (!to) return;
        if (dtype == EMB_F32) static_cast<float*>(to)[i] = s;
        else if (dtype == EMB_F16) static_cast<__half*>(to)[i] = from_float<__half>(s);
        else static_cast<__nv_bfloat16*>(to)[i] = from_float<__nv_bfloat16>(s);
    }
}

int launch(Args& a, int x_dtype, int y_dtype, bool vectors, const Shape& s, cudaStream_t st)
{
    if (!(a.status = dense_status_word())) return EMB_ERR_CUDA;
    if (x_dtype == EMB_F32) return launch_rows<float>(a, y_dtype, vectors, s, st);
    if (x_dtype == EMB_F16) return launch_rows<__half>(a, y_dtype, vectors, s, st);
    return launch_rows<__nv_bfloat16>(a, y_dtype, vectors, s, st);
}

bool params_valid(const void* weight, const void* bias, int dtype)
{
    return dtype_valid(dtype) && aligned_to(weight, dtype_bytes(dtype)) && aligned_to(bias, dtype_bytes(dtype));
}

bool eps_valid(float eps) { return eps >= 1e-24f && std::isfinite(eps); }

}  // namespace
}  // namespace norm
}  // namespace emb

using namespace emb;

extern "C" int emb_layer_norm(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t width, const void* weight,
                              const void* bias, int32_t param_dtype, float eps, void* y, int32_t y_dtype, void* stream)
{
    if (!norm::sizes_valid(rows, width) || !rows_valid(x, x_dtype, x_stride, width, rows) || !rows_valid(y, y_dtype, width, width, rows) ||
        !norm::params_valid(weight, bias, param_dtype) || !norm::eps_valid(eps))
        return EMB_ERR_INVALID_ARG;
    if (rows == 0) return EMB_OK;
    norm::Args a;
    a.x = x, a.x_stride = x_stride, a.rows = rows, a.width = (int)width;
    a.weight = weight, a.bias = bias, a.param_dtype = param_dtype, a.eps = eps, a.out = y;
    const int vector = std::min(vector_of(x, x_dtype, x_stride, width), vector_of(y, y_dtype, width, width));
    return norm::launch(a, x_dtype, y_dtype, vector == 8, norm::shape_of(rows, width, false, vector == 8), static_cast<cudaStream_t>(stream));
}

extern "C" int emb_layer_norm_grad_workspace(int64_t rows, int64_t width, size_t* bytes)
{
    if (!bytes || !norm::sizes_valid(rows, width)) return EMB_ERR_INVALID_ARG;
    const norm::Shape s = norm::shape_of(rows, width, true, true);
    const size_t need = (size_t)norm::parts_of(s) * 2 * width * sizeof(float) + norm::stats_bytes(s, rows);
    *bytes = std::max<size_t>((need + 255) & ~size_t(255), 256);
    return EMB_OK;
}

extern "C" int emb_layer_norm_grad(const void* grad_y, int32_t y_dtype, int64_t grad_stride, const void* x, int32_t x_dtype, int64_t x_stride,
                                   int64_t rows, int64_t width, const void* weight, int32_t param_dtype, float eps, void* grad_x,
                                   void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes, void* stream)
{
    size_t need = 0;
    if (emb_layer_norm_grad_workspace(rows, width, &need) != EMB_OK || !rows_valid(grad_y, y_dtype, grad_stride, width, rows) ||
        !rows_valid(x, x_dtype, x_stride, width, rows) || !rows_valid(grad_x, x_dtype, width, width, 0) ||
        !norm::params_valid(weight, nullptr, param_dtype) || !norm::params_valid(grad_weight, grad_bias, param_dtype) || !norm::eps_valid(eps) ||
        !workspace || !aligned_to(workspace, 256) || workspace_bytes < need)
        return EMB_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool params = grad_weight || grad_bias;
    if (rows == 0) {
        for (void* p : {grad_weight, grad_bias})
            if (p && cudaMemsetAsync(p, 0, (size_t)width * dtype_bytes(param_dtype), st) != cudaSuccess) return EMB_ERR_CUDA;
        return EMB_OK;
    }
    if (!params && !grad_x) return EMB_OK;
    const norm::Shape s = norm::shape_of(rows, width, true, true);
    norm::Args a;
    a.x = x, a.x_stride = x_stride, a.rows = rows, a.width = (int)width;
    a.g = grad_y, a.g_stride = grad_stride;
    a.weight = weight, a.param_dtype = param_dtype, a.eps = eps;
    a.out = grad_x, a.dw = grad_weight, a.db = grad_bias;
    if (s.kind == norm::kWideRows) a.stats = static_cast<float4*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + norm::stats_bytes(s, rows));
    int vector = std::min(vector_of(x, x_dtype, x_stride, width), vector_of(grad_y, y_dtype, grad_stride, width));
    if (grad_x) vector = std::min(vector, vector_of(grad_x, x_dtype, width, width));
    if (int rc = norm::launch(a, x_dtype, y_dtype, vector == 8, s, st)) return rc;
    const int64_t parts = norm::parts_of(s);
    if (!params || (s.kind != norm::kWideRows && parts == 1)) return EMB_OK;   // one block wrote the sums itself
    return launch_next(norm::sum_parts, dim3((unsigned)((2 * width + 31) / 32)), dim3(32, norm::kGroups), 0, st, 1, (const float*)a.partial,
                       (int)parts, (int)width, param_dtype, grad_weight, grad_bias);
}

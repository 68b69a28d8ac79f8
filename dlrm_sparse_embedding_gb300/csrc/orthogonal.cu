// Orthogonalisation of a batch of matrices by quintic Newton-Schulz steps
// (K. Jordan et al., "Muon", 2024):
//   X0 = G / (|G|_F + eps);   A = X X^T,  X <- a X + (b A + c A A) X.
//
// Three products a step.  Their operands are fp16: 11 bits where bf16 has 8, at
// the same rate.  Rounding X to fp16 would still cost much on matrices whose
// singular values fall off: the rounding of the large ones spreads over all
// directions, and every step multiplies what lies in the small ones by up to
// a.  So X is kept as the sum of two fp16 numbers (the second one scaled up, so
// that it keeps its bits where the first is subnormal), of which only the first goes
// into the products and both into the term a X: the products' part of X' lies
// in the span of the large directions, the term a X is where the small ones
// come from.  Over 128 x 256 to 1024 x 1024 matrices with flat, 1/i, 1/i^2 and
// rank-16-plus-noise spectra the result is 0.4e-3 to 1.3e-3 off the exact one
// (2-norm), below the 1.7e-3 of the output's rounding to bf16; all in bf16, it
// is 1e-2 to 1.7e-1, all in fp16 1e-3 to 2e-2.
//
// In the last two steps B = b A + c A A is stored as B + d I, and d X taken
// off again in fp32: there most singular values are near 1, B is near
// (b + c) I, and what is left of it after the shift is rounded at its own,
// smaller size.  (In earlier steps the shift would let the dropped low part of
// X back into the small directions.)
//
// Matrices whose short side m is at most kSmall go another way, in fp32: there a
// rounding has few others to average with (a 1 x 1 matrix would be 5e-3 off), and
// the work is small.  All steps are polynomials of A0 = X0 X0^T, so
//   Q = a I + b A + c A A,  A <- Q A Q,  W <- Q W,  at the end  W X0
// needs the long side only at both ends.
//
// G is scaled by a power of two before it is rounded, exact for bf16, and the
// rest of the norm goes into the first step's factors.
#include <algorithm>

#include "products.cuh"

namespace emb {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxNormBlocks = 256;   // per matrix
constexpr float kRange = 256.f;       // the scaled norm is in [kRange, 2 kRange)

struct Layout {
    int64_t ld, ldm, m, x_elems, a_elems;   // pitches (multiples of 8), the short side, elements a matrix
    int norm_blocks;
    size_t x[2], x_low[2], a, b, scale, partial, total;   // byte offsets
};

Layout layout_of(int64_t batch, int64_t rows, int64_t cols)
{
    Layout l;
    l.m = std::min(rows, cols);
    l.ld = (cols + 7) / 8 * 8;
    l.ldm = (l.m + 7) / 8 * 8;
    l.x_elems = rows * l.ld;
    l.a_elems = l.m * l.ldm;
    l.norm_blocks = (int)std::min<int64_t>(kMaxNormBlocks, (rows * cols + 8 * kNormThreads - 1) / (8 * kNormThreads));
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~size_t(255);
        return here;
    };
    for (int i = 0; i < 2; ++i) l.x[i] = take(2 * (size_t)batch * l.x_elems);
    for (int i = 0; i < 2; ++i) l.x_low[i] = take(2 * (size_t)batch * l.x_elems);
    l.a = take(2 * (size_t)batch * l.a_elems);
    l.b = take(2 * (size_t)batch * l.a_elems);
    l.scale = take(sizeof(float) * (size_t)batch);
    l.partial = take(sizeof(double) * (size_t)batch * l.norm_blocks);
    l.total = at;
    return l;
}

__device__ __forceinline__ double block_sum(double v, double* warp_sums)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0;
    for (int w = 0; w < kNormThreads / 32; ++w) s += warp_sums[w];
    return s;
}

// Calls f(row, first column, the V values there) for the elements of a matrix
// that are this warp's: rows are dealt out warp by warp, in pieces of 32 V
// columns.
template <int V, class T, class F>
__device__ __forceinline__ void each_piece(const T* g, int64_t row_stride, int64_t rows, int64_t cols, F f)
{
    constexpr int kWarps = kNormThreads / 32;
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (cols + 32 * V - 1) / (32 * V), step = (int64_t)gridDim.x * kWarps;
    int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    int64_t row = u / pieces, piece = u - row * pieces;
    const int64_t row_step = step / pieces, piece_step = step - row_step * pieces;
    while (row < rows) {
        const int64_t c = (piece * 32 + lane) * V;
        if (c < cols) {
            float v[V];
            const T* const p = g + row * row_stride + c;
            if constexpr (V == 1) {
                v[0] = to_float<T>(*p);
            } else if constexpr (sizeof(T) == 4) {
                const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            } else {
                const uint4 r = *reinterpret_cast<const uint4*>(p);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = to_float<T>(reinterpret_cast<const T*>(&r)[i]);
            }
            f(row, c, v);
        }
        row += row_step, piece += piece_step;
        if (piece >= pieces) piece -= pieces, ++row;
    }
}

// Sum of squares of each matrix, in a fixed order: fp32 within a thread, which
// has some dozens of elements, double from there.  A thread whose squares could
// leave fp32's range adds them again in double.
template <int V, class T>
__global__ void __launch_bounds__(kNormThreads) norm_partials(const T* __restrict__ g, int64_t batch_stride, int64_t row_stride,
                                                              int64_t rows, int64_t cols, double* __restrict__ partial)
{
    __shared__ double warp_sums[kNormThreads / 32];
    const T* const mine = g + blockIdx.y * batch_stride;
    float s = 0.f, top = 0.f;
    each_piece<V, T>(mine, row_stride, rows, cols, [&](int64_t, int64_t, const float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s = __fmaf_rn(v[i], v[i], s);
            top = fmaxf(top, fabsf(v[i]));
        }
    });
    double d = s;
    if (top > 1e15f || (top < 1e-15f && top > 0.f)) {
        d = 0;
        each_piece<V, T>(mine, row_stride, rows, cols, [&](int64_t, int64_t, const float (&v)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) d = fma((double)v[i], (double)v[i], d);
        });
    }
    d = block_sum(d, warp_sums);
    if (threadIdx.x == 0) partial[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = d;
}

// X = G 2^e as a sum of two fp16, and the factor that makes it G / (|G| + eps).
template <int V, class T>
__global__ void __launch_bounds__(kNormThreads) scale_in(const T* __restrict__ g, int64_t batch_stride, int64_t row_stride,
                                                         int64_t rows, int64_t cols, int norm_blocks, const double* __restrict__ partial,
                                                         float eps, int64_t ld, __half* __restrict__ x, __half* __restrict__ x_low,
                                                         float* __restrict__ scale)
{
    __shared__ double warp_sums[kNormThreads / 32];
    static_assert(kMaxNormBlocks <= kNormThreads, "one partial sum a thread");
    const double sum = block_sum(threadIdx.x < norm_blocks ? partial[(int64_t)blockIdx.y * norm_blocks + threadIdx.x] : 0.0, warp_sums);
    const double norm = sqrt(sum);
    int e = 0;
    if (norm > 0 && norm < INFINITY) e = max(-120, min(120, ilogbf(kRange) - ilogb(norm)));
    const float up = ldexpf(1.f, e);
    if (blockIdx.x == 0 && threadIdx.x == 0) scale[blockIdx.y] = (float)(1.0 / ((norm + eps) * up));
    const int64_t at = (int64_t)blockIdx.y * rows * ld;
    each_piece<V, T>(g + blockIdx.y * batch_stride, row_stride, rows, cols, [&](int64_t row, int64_t c, const float (&v)[V]) {
        alignas(16) __half h[V], l[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[i] = __float2half_rn(up * v[i]);
            l[i] = __float2half_rn(kLowScale * (up * v[i] - __half2float(h[i])));
        }
        if constexpr (V == 8) {
            *reinterpret_cast<uint4*>(x + at + row * ld + c) = *reinterpret_cast<const uint4*>(h);
            *reinterpret_cast<uint4*>(x_low + at + row * ld + c) = *reinterpret_cast<const uint4*>(l);
        } else {
            x[at + row * ld + c] = h[0];
            x_low[at + row * ld + c] = l[0];
        }
    });
}

template <int V, class T>
int start(const T* g, int64_t bs, int64_t rs, int64_t batch, int64_t rows, int64_t cols, float eps, const Layout& l, char* ws, cudaStream_t st)
{
    const dim3 grid(l.norm_blocks, (unsigned)batch);
    double* const partial = reinterpret_cast<double*>(ws + l.partial);
    norm_partials<V, T><<<grid, kNormThreads, 0, st>>>(g, bs, rs, rows, cols, partial);
    scale_in<V, T><<<grid, kNormThreads, 0, st>>>(g, bs, rs, rows, cols, l.norm_blocks, partial, eps, l.ld,
                                                  reinterpret_cast<__half*>(ws + l.x[0]), reinterpret_cast<__half*>(ws + l.x_low[0]),
                                                  reinterpret_cast<float*>(ws + l.scale));
    return cudaGetLastError() == cudaSuccess ? EMB_OK : EMB_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// short sides up to kSmall
// ---------------------------------------------------------------------------
constexpr int kSmall = 64;
constexpr int kSmallPitch = kSmall + 1;
constexpr int kSlice = 64;            // columns of the long side staged at once
constexpr int kSmallThreads = 256;
constexpr int kMaxGramBlocks = 64;    // per matrix

// Element (i, j) of the matrix with the short side first.
template <class T>
__device__ __forceinline__ float element(const T* g, int64_t row_stride, bool tall, int64_t i, int64_t j)
{
    return to_float<T>(tall ? g[j * row_stride + i] : g[i * row_stride + j]);
}

// Stage columns [j0, j0 + kSlice) of the long side, in a layout both later
// kernels read without conflicts; zeros outside the matrix.
template <class T>
__device__ __forceinline__ void stage(float (*s)[kSlice + 1], const T* g, int64_t row_stride, bool tall, int m, int64_t n, int64_t j0, float up)
{
    for (int q = threadIdx.x; q < kSmall * kSlice; q += kSmallThreads) {
        const int i = tall ? q % kSmall : q / kSlice, j = tall ? q / kSmall : q % kSlice;
        s[i][j] = i < m && j0 + j < n ? up * element<T>(g, row_stride, tall, i, j0 + j) : 0.f;
    }
    __syncthreads();
}

// One power of two for every matrix brings its largest entry near 1, so that
// no square under- or overflows.
template <class T>
__global__ void __launch_bounds__(kSmallThreads) small_largest(const T* __restrict__ g, int64_t batch_stride, int64_t row_stride,
                                                               int64_t rows, int64_t cols, unsigned* __restrict__ largest)
{
    const T* const mine = g + blockIdx.y * batch_stride;
    unsigned top = 0;   // magnitudes of floats order like their bits; NaNs come last
    for (int64_t i = (int64_t)blockIdx.x * kSmallThreads + threadIdx.x; i < rows * cols; i += (int64_t)gridDim.x * kSmallThreads)
        top = max(top, __float_as_uint(to_float<T>(mine[i / cols * row_stride + i % cols])) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) atomicMax(&largest[blockIdx.y], top);
}

__device__ __forceinline__ int small_exponent(unsigned largest)
{
    const float v = __uint_as_float(largest);
    return v > 0.f && v < INFINITY ? max(-120, min(120, -ilogbf(v))) : 0;
}

// Partial sums of G G^T (short side m) over a block's columns of the long side.
template <class T>
__global__ void __launch_bounds__(kSmallThreads) small_gram(const T* __restrict__ g, int64_t batch_stride, int64_t row_stride, bool tall, int m,
                                                            int64_t n, const unsigned* __restrict__ largest, float* __restrict__ partial)
{
    __shared__ float s[kSmall][kSlice + 1];
    const float up = ldexpf(1.f, small_exponent(largest[blockIdx.y]));
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int64_t j0 = (int64_t)blockIdx.x * kSlice; j0 < n; j0 += (int64_t)gridDim.x * kSlice) {
        stage<T>(s, g + blockIdx.y * batch_stride, row_stride, tall, m, n, j0, up);
        for (int j = 0; j < kSlice; ++j)
            for (int p = 0; p < 4; ++p)
                for (int q = 0; q < 4; ++q) acc[p][q] = __fmaf_rn(s[ti + 16 * p][j], s[tj + 16 * q][j], acc[p][q]);
        __syncthreads();
    }
    float* const to = partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kSmall * kSmall;
    for (int p = 0; p < 4; ++p)
        for (int q = 0; q < 4; ++q) to[(ti + 16 * p) * kSmall + tj + 16 * q] = acc[p][q];
}

// d = alpha * x y + beta * z + gamma * I for 64 x 64 matrices of which y is symmetric; d may be any of them.
__device__ void small_product(float* d, const float* x, const float* y, float alpha, const float* z, float beta, float gamma)
{
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int k = 0; k < kSmall; ++k)
        for (int p = 0; p < 4; ++p)
            for (int q = 0; q < 4; ++q)
                acc[p][q] = __fmaf_rn(x[(ti + 16 * p) * kSmallPitch + k], y[(tj + 16 * q) * kSmallPitch + k], acc[p][q]);
    for (int p = 0; p < 4; ++p)
        for (int q = 0; q < 4; ++q) {
            const int i = ti + 16 * p, j = tj + 16 * q;
            acc[p][q] = alpha * acc[p][q] + (z ? beta * z[i * kSmallPitch + j] : 0.f) + (i == j ? gamma : 0.f);
        }
    __syncthreads();
    for (int p = 0; p < 4; ++p)
        for (int q = 0; q < 4; ++q) d[(ti + 16 * p) * kSmallPitch + tj + 16 * q] = acc[p][q];
    __syncthreads();
}

// W, the product of all steps' Q, with the factor that takes 2^e G to X0.
__global__ void __launch_bounds__(kSmallThreads) small_steps(const float* __restrict__ partial, int parts, const unsigned* __restrict__ largest,
                                                             int m, int steps, float a, float b, float c, float eps, float* __restrict__ w_out)
{
    extern __shared__ float smem[];
    float *const A = smem, *const Q = A + kSmall * kSmallPitch, *const W = Q + kSmall * kSmallPitch;
    __shared__ float scale;
    for (int i = threadIdx.x; i < kSmall * kSmall; i += kSmallThreads) {
        float v = 0.f;
        for (int p = 0; p < parts; ++p) v += partial[((int64_t)blockIdx.x * parts + p) * kSmall * kSmall + i];
        A[i / kSmall * kSmallPitch + i % kSmall] = v;
    }
    __syncthreads();
    if (threadIdx.x == 0) {   // |2^e G|_F^2 is A's trace
        double t = 0;
        for (int i = 0; i < m; ++i) t += A[i * kSmallPitch + i];
        scale = (float)(1.0 / (sqrt(t) + (double)eps * ldexp(1.0, small_exponent(largest[blockIdx.x]))));
    }
    __syncthreads();
    const float s = scale;
    for (int i = threadIdx.x; i < kSmall * kSmallPitch; i += kSmallThreads) A[i] *= s * s;
    __syncthreads();
    for (int i = 0; i < steps; ++i) {
        small_product(Q, A, A, c, A, b, a);
        if (i == 0) {
            for (int q = threadIdx.x; q < kSmall * kSmallPitch; q += kSmallThreads) W[q] = s * Q[q];
            __syncthreads();
        } else {
            small_product(W, W, Q, 1.f, nullptr, 0.f, 0.f);
        }
        if (i + 1 < steps) {
            small_product(A, Q, A, 1.f, nullptr, 0.f, 0.f);
            small_product(A, A, Q, 1.f, nullptr, 0.f, 0.f);
        }
    }
    for (int i = threadIdx.x; i < kSmall * kSmall; i += kSmallThreads)
        w_out[(int64_t)blockIdx.x * kSmall * kSmall + i] = W[i / kSmall * kSmallPitch + i % kSmall];
}

template <class T>
__global__ void __launch_bounds__(kSmallThreads) small_apply(const T* __restrict__ g, int64_t batch_stride, int64_t row_stride, bool tall, int m,
                                                             int64_t n, const unsigned* __restrict__ largest, const float* __restrict__ w,
                                                             __nv_bfloat16* __restrict__ out)
{
    __shared__ float s[kSmall][kSlice + 1], ws[kSmall][kSmallPitch];
    const float up = ldexpf(1.f, small_exponent(largest[blockIdx.y]));
    for (int i = threadIdx.x; i < kSmall * kSmall; i += kSmallThreads) ws[i / kSmall][i % kSmall] = w[(int64_t)blockIdx.y * kSmall * kSmall + i];
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    for (int64_t j0 = (int64_t)blockIdx.x * kSlice; j0 < n; j0 += (int64_t)gridDim.x * kSlice) {
        stage<T>(s, g + blockIdx.y * batch_stride, row_stride, tall, m, n, j0, up);
        float acc[4][4] = {};
        for (int k = 0; k < kSmall; ++k)
            for (int p = 0; p < 4; ++p)
                for (int q = 0; q < 4; ++q) acc[p][q] = __fmaf_rn(ws[ti + 16 * p][k], s[k][tj + 16 * q], acc[p][q]);
        __syncthreads();
        for (int p = 0; p < 4; ++p)
            for (int q = 0; q < 4; ++q) s[ti + 16 * p][tj + 16 * q] = acc[p][q];
        __syncthreads();
        for (int q = threadIdx.x; q < kSmall * kSlice; q += kSmallThreads) {
            const int i = tall ? q % kSmall : q / kSlice, j = tall ? q / kSmall : q % kSlice;
            if (i < m && j0 + j < n) out[(int64_t)blockIdx.y * m * n + (tall ? (j0 + j) * m + i : i * n + j0 + j)] = __float2bfloat16_rn(s[i][j]);
        }
        __syncthreads();
    }
}

struct SmallLayout {
    int blocks;
    size_t largest, partial, w, total;
};

SmallLayout small_layout_of(int64_t batch, int64_t rows, int64_t cols)
{
    SmallLayout l;
    l.blocks = (int)std::min<int64_t>(kMaxGramBlocks, (std::max(rows, cols) + kSlice - 1) / kSlice);
    l.largest = 0;
    l.partial = (sizeof(unsigned) * batch + 255) & ~size_t(255);
    l.w = l.partial + sizeof(float) * (size_t)batch * l.blocks * kSmall * kSmall;
    l.total = l.w + sizeof(float) * (size_t)batch * kSmall * kSmall;
    return l;
}

template <class T>
int small(const void* update, int64_t bs, int64_t rs, int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b, float c,
          float eps, void* out, char* ws, cudaStream_t st)
{
    const SmallLayout l = small_layout_of(batch, rows, cols);
    const bool tall = rows > cols;
    const int m = (int)std::min(rows, cols);
    const int64_t n = std::max(rows, cols);
    const T* const g = static_cast<const T*>(update);
    unsigned* const largest = reinterpret_cast<unsigned*>(ws + l.largest);
    float *const partial = reinterpret_cast<float*>(ws + l.partial), *const w = reinterpret_cast<float*>(ws + l.w);
    const int smem = 3 * kSmall * kSmallPitch * (int)sizeof(float);
    const dim3 grid(l.blocks, (unsigned)batch);
    if (cudaMemsetAsync(largest, 0, sizeof(unsigned) * batch, st) != cudaSuccess ||
        cudaFuncSetAttribute(small_steps, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return EMB_ERR_CUDA;
    }
    small_largest<T><<<grid, kSmallThreads, 0, st>>>(g, bs, rs, rows, cols, largest);
    small_gram<T><<<grid, kSmallThreads, 0, st>>>(g, bs, rs, tall, m, n, largest, partial);
    small_steps<<<(unsigned)batch, kSmallThreads, smem, st>>>(partial, l.blocks, largest, m, steps, a, b, c, eps, w);
    small_apply<T><<<grid, kSmallThreads, 0, st>>>(g, bs, rs, tall, m, n, largest, w, static_cast<__nv_bfloat16*>(out));
    return cudaGetLastError() == cudaSuccess ? EMB_OK : EMB_ERR_CUDA;
}

bool sizes_valid(int64_t batch, int64_t rows, int64_t cols)
{
    return batch >= 0 && batch <= 65535 && rows >= 1 && cols >= 1 && rows <= 65536 && cols <= 65536;
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" int emb_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes)
{
    if (!bytes || !sizes_valid(batch, rows, cols)) return EMB_ERR_INVALID_ARG;
    const size_t need = std::min(rows, cols) <= kSmall ? small_layout_of(batch, rows, cols).total : layout_of(batch, rows, cols).total;
    *bytes = std::max<size_t>(256, (need + 255) & ~size_t(255));
    return EMB_OK;
}

extern "C" int emb_orthogonalize(const void* update, int32_t dtype, int64_t batch_stride, int64_t row_stride, int64_t batch,
                                 int64_t rows, int64_t cols, int32_t steps, float a, float b, float c, float eps, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    size_t need = 0;
    if (emb_orthogonalize_workspace(batch, rows, cols, &need) != EMB_OK || !dtype_valid(dtype) || steps < 1 || steps > 32 ||
        row_stride < cols || batch_stride < 0 || !aligned_to(update, dtype_bytes(dtype)) || !aligned_to(out, 2) || !(eps >= 0.f))
        return EMB_ERR_INVALID_ARG;
    if (batch == 0) return EMB_OK;
    if (!update || !out || !workspace || !aligned_to(workspace, 256) || workspace_bytes < need) return EMB_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char* const ws = static_cast<char*>(workspace);
    if (std::min(rows, cols) <= kSmall) {
        const auto go = [&](auto t) {
            return small<decltype(t)>(update, batch_stride, row_stride, batch, rows, cols, steps, a, b, c, eps, out, ws, st);
        };
        return dtype == EMB_F32 ? go(float()) : dtype == EMB_F16 ? go(__half()) : go(__nv_bfloat16());
    }
    const Layout l = layout_of(batch, rows, cols);
    const bool wide = cols % 8 == 0 && row_stride % 8 == 0 && batch_stride % 8 == 0 && aligned_to(update, 16);
    const auto begin = [&](auto t) {
        using T = decltype(t);
        const T* const g = static_cast<const T*>(update);
        return wide ? start<8, T>(g, batch_stride, row_stride, batch, rows, cols, eps, l, ws, st)
                    : start<1, T>(g, batch_stride, row_stride, batch, rows, cols, eps, l, ws, st);
    };
    int rc = dtype == EMB_F32 ? begin(float()) : dtype == EMB_F16 ? begin(__half()) : begin(__nv_bfloat16());
    const bool tall = rows > cols;
    const float* const scale = reinterpret_cast<const float*>(ws + l.scale);
    for (int i = 0; i < steps && rc == EMB_OK; ++i) {
        char *const x = ws + l.x[i & 1], *const x_low = ws + l.x_low[i & 1];
        const float d = i == 0 ? 0.f : i == steps - 1 ? -0.9f * (b + c) : i == steps - 2 ? -0.73f * (b + c) : 0.f;
        ProductArgs s;   // A = X X^T, or X^T X
        s.batch = batch;
        s.a = s.b = x, s.lda = s.ldb = l.ld, s.batch_a = s.batch_b = l.x_elems;
        s.a_mn = s.b_mn = tall;
        s.m = s.n = l.m, s.k = std::max(rows, cols);
        if (i == 0) s.scale = scale;
        s.d = ws + l.a, s.ldd = l.ldm, s.batch_d = l.a_elems;
        rc = launch_product(s, st);
        if (rc != EMB_OK) break;
        ProductArgs q;   // B = c A A + b A + d I
        q.batch = batch;
        q.a = q.b = q.c = ws + l.a, q.lda = q.ldb = q.ldc = l.ldm, q.batch_a = q.batch_b = q.batch_c = l.a_elems;
        q.m = q.n = q.k = l.m;
        q.alpha = c, q.beta = b, q.diagonal = d;
        q.d = ws + l.b, q.ldd = l.ldm, q.batch_d = l.a_elems;
        rc = launch_product(q, st);
        if (rc != EMB_OK) break;
        ProductArgs n;   // X <- (a - d) X + B X, or X B
        n.batch = batch;
        n.a = tall ? x : ws + l.b, n.lda = tall ? l.ld : l.ldm, n.batch_a = tall ? l.x_elems : l.a_elems;
        n.b = tall ? ws + l.b : x, n.ldb = tall ? l.ldm : l.ld, n.batch_b = tall ? l.a_elems : l.x_elems;
        n.b_mn = !tall;
        n.m = rows, n.n = cols, n.k = l.m;
        if (i == 0) n.scale = scale;
        n.beta = a - d, n.c = x, n.c_low = x_low, n.ldc = l.ld, n.batch_c = l.x_elems;
        if (i == steps - 1) {
            n.d = out, n.d_dtype = EMB_BF16, n.ldd = cols, n.batch_d = rows * cols;
        } else {
            n.d = ws + l.x[(i + 1) & 1], n.d_low = ws + l.x_low[(i + 1) & 1], n.ldd = l.ld, n.batch_d = l.x_elems;
        }
        rc = launch_product(n, st);
    }
    return rc;
}

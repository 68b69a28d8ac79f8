// Layer norm of rows and its gradients.
//
//   h = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  y = h w + b
//   dx = rstd (g w - mean(g w) - h mean(g w h)),  dw = sum over rows of g h,  db = sum over rows of g
//
// Bound by memory: x (and g) is read once and y (dx) written once.  A row's elements
// stay in the registers of the threads that share it, so the mean, the variance
// around it and the result are three passes over registers.  The gradient takes x
// again instead of stored statistics: it has to read x for h, and the two sums more
// hide behind the loads of the next row.
//
// The mean is a rounded sum; what the rounding left, d = mean(x - m), is measured in the
// second pass and taken off again, so rows far from zero lose no more than their own
// rounding.  Where squares leave fp32's range (|x| of 2^50 and more) the row is
// taken again times 2^-80.
//
// dw and db: a block walks many rows and its threads add up their own columns in
// registers; the blocks' sums go to the workspace and a second kernel adds them in a
// fixed order, so results repeat bit for bit.
#pragma once

#include "rows.cuh"

namespace emb {
namespace norm {

struct Args {
    const void* x = nullptr;
    const void* g = nullptr;       // gradient of y (null: forward)
    int64_t x_stride = 0, g_stride = 0, rows = 0;
    int width = 0;
    const void* weight = nullptr;  // null: ones
    const void* bias = nullptr;    // null: zeros
    int param_dtype = EMB_F32;
    float eps = 0.f;
    void* out = nullptr;           // y, or dx (nullable), contiguous
    void* dw = nullptr;            // nullable
    void* db = nullptr;            // nullable
    float* partial = nullptr;      // [blocks][2][width]
    float4* stats = nullptr;       // of each row, wide rows only: m, d, rstd, scale
};

// How the rows are laid on the grid.
struct Shape {
    int per_thread;        // elements of a row a thread holds: 8 or 16, or 0 for wide rows
    int tx, ty;            // threads a row (up to a warp, or several and then ty is 1); rows a block
    int blocks;
    int chunks;            // wide rows' gradients: parts the rows are added up in
};

constexpr int kThreads = 256, kMaxThreads = 512, kWideThreads = 1024;
constexpr int kRegisterWidth = 16 * kMaxThreads;   // the widest row kept in registers
// Registers a thread: what its elements take (16 of a gradient spill a few words).
constexpr int registers(int per_thread, bool grad) { return per_thread == 16 ? 128 : grad ? 80 : 64; }
constexpr int kColumnRows = 8;              // rows at a time of a block of wide_columns

// int launch(const Args&, x type, out type, g type ...): one translation unit for each type of x
template <class X> int launch_rows(const Args& a, int y_dtype, int vector, const Shape& s, cudaStream_t st);

#ifdef EMB_NORM_KERNELS

__device__ __forceinline__ float param(const void* p, int dtype, int64_t i, float none)
{
    if (!p) return none;
    if (dtype == EMB_F32) return __ldg(static_cast<const float*>(p) + i);
    if (dtype == EMB_F16) return __half2float(__ldg(static_cast<const __half*>(p) + i));
    return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}

__device__ __forceinline__ void store_param(void* p, int dtype, int64_t i, float v)
{
    if (!p) return;
    if (dtype == EMB_F32) static_cast<float*>(p)[i] = v;
    else if (dtype == EMB_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// s, summed over the blockDim.x threads of a row, in all of them.  Two calls in turn
// on two buffers need no barrier more: the other call's lies between.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*part)[4])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = 16; d; d >>= 1)
            if (d < blockDim.x) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
    if (blockDim.x <= 32) return;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[threadIdx.x >> 5][i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
    for (int v = 0; v < warps; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += part[v][i];
}

// Squares up to here are summed as they are; a row beyond is scaled.
constexpr float kLargeSquares = 0x1p100f, kDown = 0x1p-80f;

struct Moments {
    float m, d, rstd, scale;
    __device__ __forceinline__ float h(float x) const { return ((x * scale - m) - d) * rstd; }
};

__device__ __forceinline__ Moments moments(float m, float shifted, float squares, float inv_n, float eps, float scale)
{
    Moments r;
    r.m = m;
    r.d = shifted * inv_n;
    const float var = fmaxf(squares * inv_n - r.d * r.d, 0.f) + eps * scale * scale;
    // fmaxf drops a NaN: rows that hold one, or an infinity, are NaN all over
    r.rstd = squares == squares ? (var > 0.f ? 1.f / sqrtf(var) : 0.f) : squares;
    r.scale = scale;
    return r;
}

// Rows of up to kRegisterWidth elements: U vectors of V a thread.
template <int V, int U, bool GRAD, class X, class Y>
__global__ void __maxnreg__(registers(U * V, GRAD)) norm_rows(const Args a)
{
    __shared__ float part[2][32][4];
    extern __shared__ float dynamic[];
    let_next_begin();
    wait_for_earlier();
    const int tx = threadIdx.x, width = a.width;
    const float inv_n = 1.f / (float)width;
    const X* const x = static_cast<const X*>(a.x);
    const Y* const g = static_cast<const Y*>(a.g);
    const auto column = [&](int u) { return (tx + u * (int)blockDim.x) * V; };

    float w[U][V], b[U][V], acc_w[U][V], acc_b[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const bool in = column(u) < width;
            w[u][q] = in ? param(a.weight, a.param_dtype, column(u) + q, 1.f) : 0.f;
            if (!GRAD) b[u][q] = in ? param(a.bias, a.param_dtype, column(u) + q, 0.f) : 0.f;
            acc_w[u][q] = acc_b[u][q] = 0.f;
        }

    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    Raw<V, X> next_x[U];
    Raw<V, Y> next_g[U];
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row < a.rows && column(u) < width) {
                next_x[u].load(x + row * a.x_stride + column(u));
                if (GRAD) next_g[u].load(g + row * a.g_stride + column(u));
            }
    };
    int64_t first = (int64_t)blockIdx.x * blockDim.y;
    fetch(first + threadIdx.y);
    // a block's rows move on together: every thread meets every barrier
    for (; first < a.rows; first += step) {
        const int64_t row = first + threadIdx.y;
        const bool has = row < a.rows;
        float v[U][V], gr[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const bool in = has && column(u) < width;
                v[u][q] = in ? next_x[u][q] : 0.f;
                if (GRAD) gr[u][q] = in ? next_g[u][q] : 0.f;
            }
        fetch(row + step);

        Moments mo;
        float along = 0.f, mean_gw = 0.f;
        float scale = 1.f;
        for (bool again = false;; again = true) {
            float s1[1] = {};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int q = 0; q < V; ++q) s1[0] += v[u][q] * scale;
            row_sums<1>(s1, part[0]);
            const float m = s1[0] * inv_n;
            float s[GRAD ? 4 : 2] = {};
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (column(u) < width) {
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const float c = v[u][q] * scale - m;
                        s[0] += c;
                        s[1] = __fmaf_rn(c, c, s[1]);
                        if constexpr (GRAD) {
                            const float gw = gr[u][q] * w[u][q];
                            s[2] += gw;
                            s[3] = __fmaf_rn(gw, c, s[3]);
                        }
                    }
                }
            row_sums<GRAD ? 4 : 2>(s, part[1]);
            const bool large = !(s[1] <= kLargeSquares);
            if (!again && __any_sync(0xffffffffu, large)) {   // the same in all threads of a row, and in all that meet a barrier
                scale = large ? kDown : 1.f;
                continue;
            }
            mo = moments(m, s[0], s[1], inv_n, a.eps, scale);
            if constexpr (GRAD) {
                mean_gw = s[2] * inv_n;
                along = (s[3] - mo.d * s[2]) * mo.rstd * inv_n;
            }
            break;
        }
        const float outer = mo.rstd * mo.scale;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float o[V];
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float h = mo.h(v[u][q]);
                if constexpr (GRAD) {
                    acc_w[u][q] = __fmaf_rn(gr[u][q], h, acc_w[u][q]);
                    acc_b[u][q] += gr[u][q];
                    o[q] = outer * ((gr[u][q] * w[u][q] - mean_gw) - h * along);
                } else {
                    o[q] = __fmaf_rn(h, w[u][q], b[u][q]);
                }
            }
            if (has && column(u) < width && a.out) {
                if constexpr (GRAD) store_vec<V, X>(static_cast<X*>(a.out) + row * width + column(u), o);
                else store_vec<V, Y>(static_cast<Y*>(a.out) + row * width + column(u), o);
            }
        }
    }
    if constexpr (GRAD) {
        if (!a.dw && !a.db) return;
        const auto put = [&](int which, int c, float sum) {
            if (gridDim.x == 1) store_param(which ? a.db : a.dw, a.param_dtype, c, sum);
            else a.partial[((int64_t)blockIdx.x * 2 + which) * width + c] = sum;
        };
        for (int which = 0; which < 2; ++which) {
            if (blockDim.y > 1) {   // the block's rows meet: dynamic[ty][column]
                const int cols = (int)blockDim.x * U * V;
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < V; ++q) dynamic[threadIdx.y * cols + column(u) + q] = which ? acc_b[u][q] : acc_w[u][q];
                __syncthreads();
                for (int c = threadIdx.y * blockDim.x + tx; c < width; c += blockDim.x * blockDim.y) {
                    float sum = 0.f;
                    for (int r = 0; r < blockDim.y; ++r) sum += dynamic[r * cols + c];
                    put(which, c, sum);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (column(u) < width) {
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            put(which, column(u) + q, which ? acc_b[u][q] : acc_w[u][q]);
                    }
            }
        }
    }
}

// Wider rows: a block takes one, three times over, the later ones from the caches.
template <int V, bool GRAD, class X, class Y>
__global__ void __launch_bounds__(kWideThreads) wide_rows(const Args a)
{
    __shared__ float part[2][32][4];
    let_next_begin();
    wait_for_earlier();
    const int width = a.width, step = (int)blockDim.x * V;
    const float inv_n = 1.f / (float)width;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const X* const x = static_cast<const X*>(a.x) + row * a.x_stride;
        const Y* const g = static_cast<const Y*>(a.g) + row * a.g_stride;
        Moments mo;
        float along = 0.f, mean_gw = 0.f, scale = 1.f;
        for (bool again = false;; again = true) {
            float s1[1] = {};
            for (int c = threadIdx.x * V; c < width; c += step) {
                Raw<V, X> v;
                v.load(x + c);
#pragma unroll
                for (int q = 0; q < V; ++q) s1[0] += v[q] * scale;
            }
            row_sums<1>(s1, part[0]);
            const float m = s1[0] * inv_n;
            float s[GRAD ? 4 : 2] = {};
            for (int c = threadIdx.x * V; c < width; c += step) {
                Raw<V, X> v;
                Raw<V, Y> gr;
                v.load(x + c);
                if (GRAD) gr.load(g + c);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float e = v[q] * scale - m;
                    s[0] += e;
                    s[1] = __fmaf_rn(e, e, s[1]);
                    if constexpr (GRAD) {
                        const float gw = gr[q] * param(a.weight, a.param_dtype, c + q, 1.f);
                        s[2] += gw;
                        s[3] = __fmaf_rn(gw, e, s[3]);
                    }
                }
            }
            row_sums<GRAD ? 4 : 2>(s, part[1]);
            if (!again && !(s[1] <= kLargeSquares)) {
                scale = kDown;
                continue;
            }
            mo = moments(m, s[0], s[1], inv_n, a.eps, scale);
            if constexpr (GRAD) {
                mean_gw = s[2] * inv_n;
                along = (s[3] - mo.d * s[2]) * mo.rstd * inv_n;
            }
            break;
        }
        if (GRAD && a.stats && threadIdx.x == 0) a.stats[row] = make_float4(mo.m, mo.d, mo.rstd, mo.scale);
        if (!a.out) continue;
        const float outer = mo.rstd * mo.scale;
        for (int c = threadIdx.x * V; c < width; c += step) {
            Raw<V, X> v;
            Raw<V, Y> gr;
            float o[V];
            v.load(x + c);
            if (GRAD) gr.load(g + c);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float h = mo.h(v[q]), w = param(a.weight, a.param_dtype, c + q, 1.f);
                if constexpr (GRAD) o[q] = outer * ((gr[q] * w - mean_gw) - h * along);
                else o[q] = __fmaf_rn(h, w, param(a.bias, a.param_dtype, c + q, 0.f));
            }
            if constexpr (GRAD) store_vec<V, X>(static_cast<X*>(a.out) + row * width + c, o);
            else store_vec<V, Y>(static_cast<Y*>(a.out) + row * width + c, o);
        }
    }
}

// The column sums of wide rows' gradients: a warp has 32 vectors' columns, a block
// kColumnRows rows at a time of its part of the rows.
template <int V, class X, class Y>
__global__ void __launch_bounds__(32 * kColumnRows) wide_columns(const Args a)
{
    __shared__ float sums[kColumnRows][32 * V];
    let_next_begin();
    wait_for_earlier();
    const int width = a.width, lane = threadIdx.x, c = (blockIdx.x * 32 + lane) * V;
    float acc_w[V] = {}, acc_b[V] = {};
    if (c < width)
        for (int64_t row = (int64_t)blockIdx.y * kColumnRows + threadIdx.y; row < a.rows; row += (int64_t)gridDim.y * kColumnRows) {
            const float4 st = a.stats[row];
            const Moments mo{st.x, st.y, st.z, st.w};
            Raw<V, X> v;
            Raw<V, Y> g;
            v.load(static_cast<const X*>(a.x) + row * a.x_stride + c);
            g.load(static_cast<const Y*>(a.g) + row * a.g_stride + c);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                acc_w[q] = __fmaf_rn(g[q], mo.h(v[q]), acc_w[q]);
                acc_b[q] += g[q];
            }
        }
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < V; ++q) sums[threadIdx.y][lane * V + q] = which ? acc_b[q] : acc_w[q];
        __syncthreads();
        for (int i = threadIdx.y * 32 + lane; i < 32 * V; i += 32 * kColumnRows) {
            const int col = blockIdx.x * 32 * V + i;
            if (col >= width) continue;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < kColumnRows; ++r) s += sums[r][i];
            a.partial[((int64_t)blockIdx.y * 2 + which) * width + col] = s;
        }
    }
}

template <class X>
int launch_rows(const Args& a, int y_dtype, int vector, const Shape& s, cudaStream_t st)
{
    return with_type(y_dtype, [&](auto yt) {
        using Y = decltype(yt);
        const auto go = [&](auto v, auto grad) {
            constexpr int V = decltype(v)::value;
            constexpr bool GRAD = decltype(grad)::value;
            const dim3 block(s.tx, s.ty);
            if (!s.per_thread) {
                if (int rc = launch_next(wide_rows<V, GRAD, X, Y>, s.blocks, kWideThreads, 0, st, 1, a)) return rc;
                if constexpr (GRAD) {
                    if (a.dw || a.db)
                        return launch_next(wide_columns<V, X, Y>, dim3((a.width + 32 * V - 1) / (32 * V), s.chunks), dim3(32, kColumnRows), 0, st, 1, a);
                }
                return (int)EMB_OK;
            }
            const size_t smem = GRAD && s.ty > 1 ? (size_t)s.tx * s.ty * s.per_thread * sizeof(float) : 0;
            return launch_next(s.per_thread == 8 ? norm_rows<V, 8 / V, GRAD, X, Y> : norm_rows<V, 16 / V, GRAD, X, Y>,
                               s.blocks, block, smem, st, 1, a);
        };
        const auto with_v = [&](auto grad) {
            return vector == 8 ? go(std::integral_constant<int, 8>(), grad) : go(std::integral_constant<int, 1>(), grad);
        };
        return a.g ? with_v(std::true_type()) : with_v(std::false_type());
    });
}

#endif  // EMB_NORM_KERNELS

}  // namespace norm
}  // namespace emb

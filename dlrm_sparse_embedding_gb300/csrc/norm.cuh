// Layer norm of rows and its gradients.
//
//   h = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  y = h w + b
//   dx = rstd (g w - mean(g w) - h mean(g w h)),  dw = sum over rows of g h,  db = sum over rows of g
//
// Bound by memory: x (and g) is read once and y (dx) written once.  Rows come to shared
// memory by bulk copies through a ring of stages, so what is on its way costs no registers, and
// from there once to the registers of the threads that share the row; the mean, the variance
// around it and the result are three passes over registers.  The gradient takes x again instead of
// stored statistics: it has to read x for h.  fp32 elements take two an instruction.
//
// 16384 x 3328, fp32 to bf16: forward 51 us (6.5 TB/s), gradients 87 (6.3).  Two bytes an element are too
// few for the sums' latency and instructions: bf16 alone 42 (5.2 TB/s) and 86 (3.8); 425984 x 128
// bf16 39 (5.7) and 67 (4.9).  Rows without a 16-byte rhythm go element by element: 32768 x 1025 fp16 81
// and 94 us (1.7 and 2.1), and their kernels spill 16 to 100 bytes a thread (a warp's rows of 32 elements a thread
// up to 184).  Past 8192 elements (of a forward in vectors, 16384) a row is read three times
// and its columns' sums by a second kernel: 4000 x 16384 gradients fp32 to bf16 305 us (2.1), bf16 194 (2.0);
// 2000 x 32768 forward 191 (2.1) and 128 (2.1).
//
// The mean is a rounded sum; what the rounding left, d = mean(x - m), is measured in the
// second pass and taken off again, so rows far from zero lose no more than their own
// rounding.  Where squares leave fp32's range (|x| of 2^50 and more) the row is
// taken again times 2^-80.
//
// dw and db: a block walks many rows and its threads add up their own columns in
// registers; the blocks' sums go to the workspace and a second kernel adds them in a
// fixed order, so results repeat bit for bit.
//
// Measured and not kept: rows by loads into registers a row ahead (333 us for the first line's 143);
// eight elements a thread (forward 65, gradients 102); statistics around the mean of 32 samples, a barrier
// less, whose second try for rows they do not fit costs registers (bf16 gradients 85 us, but
// fp32's 101); short rows' parameters in shared memory, for more warps (42 and 84 us where 39 and 70); rows
// past 8192 shared by a cluster's blocks (307 us).
#pragma once

#include <algorithm>
#include <atomic>

#include "emb_internal.cuh"
#include "rows.cuh"
#include "tensor_core.cuh"

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
    int* status = nullptr;
    // the ring of stages that rows are copied to
    int stages = 0, chunk = 1;     // rows of a stage
    bool x_whole = false, g_whole = false;   // a stage's rows are one piece of memory
    int x_pitch = 0, g_pitch = 0;  // bytes between a stage's rows in shared memory, where they are not
    int x_slot = 0, g_slot = 0;    // bytes of a stage
};

// How rows are laid on the grid.
enum Kind { kWarpRows, kBlockRows, kWideRows };
struct Shape {
    Kind kind;
    int tx, ty;            // threads a row; rows a block
    int per_thread;        // elements of a row a thread holds
    int blocks, per_sm;
    int chunks;            // wide rows' gradients: parts the rows are added up in
};

constexpr int kThreads = 256, kMaxThreads = 512, kWideThreads = 512;
// Elements of a row a thread holds: 16, and 32 of longer rows where only the forward's two
// parameters are held beside them and elements come in vectors.
constexpr int kFew = 16, kMany = 32;
constexpr int kMaxStages = 8, kMaxSubs = 5;
constexpr int kSharedBytes = 226 * 1024;         // of an SM, for its blocks
constexpr int kOwnBytes = 2944;                  // of a block beside its stages
// Of an SM, for the stages, two at least: more on their way are slower (16384 x 3328, fp32 to bf16, forward:
// 51 us, with all of the memory 58; gradients 86 and 87, with two stages 94).
constexpr int kRingBytes = 120 * 1024;
constexpr int kChunkBytes = 4096;                // of a warp's stage
constexpr int kColumnRows = 8;                   // rows at a time of a block of wide_columns
// Registers a thread: what its elements take.
constexpr int registers(int per_thread, bool grad, bool vectors) { return grad || per_thread == kMany ? 128 : vectors ? 80 : 96; }

// One translation unit for each type of x.  `vectors`: rows of both types are whole
// vectors, all at 16-byte boundaries.
template <class X> int launch_rows(Args a, int y_dtype, bool vectors, const Shape& s, cudaStream_t st);

#ifdef EMB_NORM_KERNELS

__device__ __forceinline__ float param(const void* p, int dtype, int64_t i, float none)
{
    if (!p) return none;
    if (dtype == EMB_F32) return __ldg(static_cast<const float*>(p) + i);
    if (dtype == EMB_F16) return __half2float(__ldg(static_cast<const __half*>(p) + i));
    return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}

// V of them from i on, a vector where they are at its boundary.
template <int V>
__device__ __forceinline__ void params(const void* p, int dtype, int64_t i, float none, float (&to)[V])
{
    if (V > 1 && p && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const auto get = [&](auto t) {
            using T = decltype(t);
            Raw<V, T> r;
            r.load_again(static_cast<const T*>(p) + i);
#pragma unroll
            for (int q = 0; q < V; ++q) to[q] = r[q];
        };
        if (dtype == EMB_F32) get(float());
        else if (dtype == EMB_F16) get(__half());
        else get(__nv_bfloat16());
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q) to[q] = param(p, dtype, i + q, none);
    }
}

__device__ __forceinline__ void store_param(void* p, int dtype, int64_t i, float v)
{
    if (!p) return;
    if (dtype == EMB_F32) static_cast<float*>(p)[i] = v;
    else if (dtype == EMB_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// s, summed over `lanes` lanes (a power of two), in all of them.  The lanes first share the
// values out, each half of them going on with half of the values, so that N values
// take N - 1 + log2(lanes / N) exchanges and N to hand them back instead of N log2(lanes).
template <int N>
__device__ __forceinline__ void lane_sums(float (&s)[N], int lanes)
{
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x + threadIdx.y * blockDim.x;
    if (N == 1 || lanes < 2 * N) {
#pragma unroll
        for (int d = 16; d; d >>= 1)
            if (d < lanes)
#pragma unroll
                for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(kAll, s[i], d);
        return;
    }
    float v = 0.f;
    if constexpr (N == 4) {
        const bool up = lane & 2, odd = lane & 1;
        float p = up ? s[2] : s[0], q = up ? s[3] : s[1];
        p += __shfl_xor_sync(kAll, up ? s[0] : s[2], 2);
        q += __shfl_xor_sync(kAll, up ? s[1] : s[3], 2);
        v = (odd ? q : p) + __shfl_xor_sync(kAll, odd ? p : q, 1);
    } else if constexpr (N == 2) {
        const bool odd = lane & 1;
        v = (odd ? s[1] : s[0]) + __shfl_xor_sync(kAll, odd ? s[0] : s[1], 1);
    }
#pragma unroll
    for (int d = 16; d >= N; d >>= 1)
        if (d < lanes) v += __shfl_xor_sync(kAll, v, d);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __shfl_sync(kAll, v, (lane & 31 & ~(N - 1)) | i);   // value i is lane i's of every N
}

// The same over the blockDim.x threads (at most 16 warps) of a row, of which a block may have
// several: row `sub`'s threads meet at a barrier of their own.  Two calls in turn on two
// buffers need no barrier more: the other call's lies between.
template <int N, bool SUBS>
__device__ __forceinline__ void block_sums(float (&s)[N], float (*part)[4], int sub)
{
    lane_sums(s, 32);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[threadIdx.x >> 5][i] = s[i];
    if constexpr (SUBS) asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(blockDim.x) : "memory");
    else __syncthreads();
    // lane (w, i) adds up warps w, w + 32 / N, ...
    const int i = lane & (N - 1);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; w += 32 / N)
        if (w + lane / N < warps) v += part[w + lane / N][i];
#pragma unroll
    for (int d = 16; d >= N; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = __shfl_sync(0xffffffffu, v, (lane & ~(N - 1)) | j);
}

// Two fp32 numbers that one instruction takes.
struct Two {
    uint64_t bits;
    __device__ __forceinline__ Two() = default;
    __device__ __forceinline__ Two(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(x), "f"(y)); }
    __device__ __forceinline__ explicit Two(float x) : Two(x, x) {}
    __device__ __forceinline__ float2 both() const
    {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(bits));
        return r;
    }
};
__device__ __forceinline__ Two operator+(Two a, Two b)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits));
    return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits));
    return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
    return r;
}
__device__ __forceinline__ float sum(Two a) { const float2 v = a.both(); return v.x + v.y; }

// Squares up to here are summed as they are; a row beyond is scaled.
constexpr float kLargeSquares = 0x1p100f, kDown = 0x1p-80f;

struct Moments {
    float m, d, rstd, scale;
    __device__ __forceinline__ float h(float x) const { return __fmaf_rn(x * scale - m, rstd, -d * rstd); }
};

// 1 / sqrt(v): the approximation and one step of Newton's method, within 2^-23.
__device__ __forceinline__ float root(float v)
{
    const float r = rsqrtf(v);
    return __fmaf_rn(0.5f * r, __fmaf_rn(-v * r, r, 1.f), r);
}

__device__ __forceinline__ Moments moments(float m, float shifted, float squares, float inv_n, float eps, float scale)
{
    Moments r;
    r.m = m;
    r.d = shifted * inv_n;
    const float var = fmaxf(squares * inv_n - r.d * r.d, 0.f) + eps * scale * scale;
    // fmaxf drops a NaN: rows that hold one, or an infinity, are NaN all over
    r.rstd = squares == squares ? (var > 0.f ? root(var) : 0.f) : squares;
    r.scale = scale;
    return r;
}

// What a thread holds of a row, U vectors of V, and adds up over rows.
template <int V, int U, bool GRAD, bool BLOCK, class X, class Y>
struct Piece {
    static constexpr int E = U * V;
    Two v[E / 2], g[E / 2], w[E / 2], b[E / 2], acc_w[E / 2], acc_b[E / 2];
    int first, step, width;    // its columns: V from first + u * step on

    __device__ __forceinline__ bool in(int u) const { return first + u * step < width; }

    // A parameter's elements, all of them on their way before the first is used.
    __device__ __forceinline__ void fill(const void* p, int dtype, float none, Two (&to)[E / 2])
    {
        float t[E];
        const auto get = [&](auto as) {
            using T = decltype(as);
            const T* const from = static_cast<const T*>(p) + first;
            if (V > 1 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                Raw<V, T> r[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    r[u].clear();
                    if (in(u)) r[u].load_again(from + u * step);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] = r[e / V][e % V];
            } else {
                Raw<1, T> r[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    r[e].clear();
                    if (in(e / V)) r[e].load_again(from + e / V * step + e % V);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] = r[e][0];
            }
        };
        if (!p) {
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = in(e / V) ? none : 0.f;
        } else if (dtype == EMB_F32) get(float());
        else if (dtype == EMB_F16) get(__half());
        else get(__nv_bfloat16());
#pragma unroll
        for (int e = 0; e < E; e += 2) to[e / 2] = Two(t[e], t[e + 1]);
    }

    __device__ __forceinline__ void open(const Args& a, int tx, int threads)
    {
        first = tx * V, step = threads * V, width = a.width;
        fill(a.weight, a.param_dtype, 1.f, w);
        if (!GRAD) fill(a.bias, a.param_dtype, 0.f, b);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) acc_w[i] = acc_b[i] = Two(0.f);
    }

    template <class T>
    __device__ __forceinline__ void take(const T* p, bool has, Two (&to)[E / 2])
    {
        Raw<V, T> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u].clear();
            if (has && in(u)) r[u].load_shared(p + first + u * step);
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) to[e / 2] = Two(r[e / V][e % V], r[(e + 1) / V][(e + 1) % V]);
    }

    // A row in shared memory, and its results to where() (null: nowhere).  first_sums and
    // second_sums add up over the row's threads; any(flag) tells whether a row's of all
    // that add up together is set.
    using O = typename std::conditional<GRAD, X, Y>::type;
    template <class WHERE, class S1, class S2, class ANY>
    __device__ __forceinline__ void row(const Args& a, const X* x, const Y* gy, WHERE where, bool has, float inv_n, S1 first_sums, S2 second_sums, ANY any)
    {
        constexpr int N = GRAD ? 4 : 2;
        take(x, has, v);
        if constexpr (GRAD) take(gy, has, g);
        Moments mo;
        float scale = 1.f, s[N];
        for (;;) {
            Two t = v[0];
#pragma unroll
            for (int i = 1; i < E / 2; ++i) t = t + v[i];
            float s1[1] = {sum(t)};
            first_sums(s1);
            mo.m = s1[0] * inv_n;
            Two s0(0.f), sq(0.f), sg(0.f), sgc(0.f);
            const auto add = [&](int i) {
                s0 = s0 + v[i];
                sq = fma(v[i], v[i], sq);
                if constexpr (GRAD) {
                    const Two gw = g[i] * w[i];
                    sg = sg + gw;
                    sgc = fma(gw, v[i], sgc);
                }
            };
            if constexpr (V > 1) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // where there is nothing, zero stays zero; a block's gradient is faster without the
                    // branch (16384 x 3328, fp32 to bf16: 98 and 87 us), a warp's with it (425984 x 128: 93 and 105)
                    const Two less(in(u) ? -mo.m : 0.f);
                    if (!BLOCK && !in(u)) continue;
#pragma unroll
                    for (int i = u * V / 2; i < (u + 1) * V / 2; ++i) {
                        v[i] = v[i] + less;
                        add(i);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const float2 c = (v[i] + Two(-mo.m)).both();
                    v[i] = Two(in(2 * i) ? c.x : 0.f, in(2 * i + 1) ? c.y : 0.f);
                    add(i);
                }
            }
            s[0] = sum(s0), s[1] = sum(sq);
            if constexpr (GRAD) s[2] = sum(sg), s[3] = sum(sgc);
            second_sums(s);
            const bool large = scale == 1.f && !(s[1] <= kLargeSquares);
            if (!any(large)) break;
            // once more, those rows smaller
            if (large) scale = kDown;
            take(x, has, v);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = v[i] * Two(scale);
        }
        mo = moments(mo.m, s[0], s[1], inv_n, a.eps, scale);
        const Two rstd(mo.rstd), shift(-mo.d * mo.rstd);
        Two k1, k2, k3;     // dx = k1 g w + k2 h + k3
        if constexpr (GRAD) {
            const float k = mo.rstd * scale;
            k1 = Two(k);
            k2 = Two(-k * ((s[3] - mo.d * s[2]) * mo.rstd * inv_n));
            k3 = Two(-k * (s[2] * inv_n));
        }
        float o[E];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const Two h = fma(v[i], rstd, shift);
            Two r;
            if constexpr (GRAD) {
                acc_w[i] = fma(g[i], h, acc_w[i]);
                acc_b[i] = acc_b[i] + g[i];
                r = fma(g[i] * w[i], k1, fma(h, k2, k3));
            } else {
                r = fma(h, w[i], b[i]);
            }
            const float2 both = r.both();
            o[2 * i] = both.x, o[2 * i + 1] = both.y;
        }
        O* const out = where();
        if (!has || !out) return;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (in(u)) store_vec<V, O>(out + first + u * step, reinterpret_cast<const float(&)[V]>(o[u * V]));
    }

    __device__ __forceinline__ float sum_of(int which, int e) const
    {
        const float2 both = (which ? acc_b[e / 2] : acc_w[e / 2]).both();
        return e & 1 ? both.y : both.x;
    }
};

// Where `bytes` at p lie between 16-byte boundaries.
struct Span {
    const unsigned char* from;
    uint32_t bytes, skip;
    __device__ __forceinline__ Span(const void* p, int64_t n)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), begin = at & ~uintptr_t(15);
        from = reinterpret_cast<const unsigned char*>(begin);
        skip = (uint32_t)(at - begin);
        bytes = (uint32_t)((at + n + 15 - begin) & ~uintptr_t(15));
    }
};

// If a wait gave up, what was copied last lands before the block ends.
__device__ __forceinline__ void gave_up_end(int* status)
{
    const uint64_t t0 = tc::now_ns();
    while (tc::now_ns() - t0 < 2000000) {}
    if (status) atomicOr(status, ERRBIT_TIMEOUT);
}

// The sums of a block's threads, which take up to blockDim.y rows at a time: to its part
// of the workspace, or, of a block alone, to their place.
template <class PIECE, int V, int U>
__device__ __forceinline__ void put_sums(const Args& a, const PIECE& p, float* shared, int ty)
{
    const auto put = [&](int which, int c, float sum) {
        if (gridDim.x == 1) store_param(which ? a.db : a.dw, a.param_dtype, c, sum);
        else a.partial[((int64_t)blockIdx.x * 2 + which) * a.width + c] = sum;
    };
    const int threads = blockDim.x * blockDim.y, thread = threadIdx.y * blockDim.x + threadIdx.x, cols = p.step * U;
    for (int which = 0; which < 2; ++which) {
        if (ty > 1) {   // the rows meet: shared[row][column]
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int q = 0; q < V; ++q) shared[threadIdx.y * cols + p.first + u * p.step + q] = p.sum_of(which, u * V + q);
            __syncthreads();
            for (int c = thread; c < a.width; c += threads) {
                float sum = 0.f;
                for (int r = 0; r < ty; ++r) sum += shared[r * cols + c];
                put(which, c, sum);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p.in(u)) {
#pragma unroll
                    for (int q = 0; q < V; ++q) put(which, p.first + u * p.step + q, p.sum_of(which, u * V + q));
                }
        }
    }
}

// Longer rows: blockDim.x threads take one at a time, and a block has, SUBS, up to kMaxSubs rows'
// threads, so that fewer blocks leave sums of a gradient's columns (1000 x 1024 bf16: 19.0 us with
// one, 8.6 with four; 50000: 74.0 and 71.4).  Rows are
// copied to a ring of stages, each row's threads have their own; a stage is free for the
// next row when the second sums' barrier has been met.
//
// Each thread waits for itself, and one whose wait gave up goes on to the barriers, since the
// row's other threads count on it.  Between the row's two barriers nobody waits: there they say
// in `leave` what they all read behind the second one, to write nothing and leave together.  (What each keeps
// of it in a register instead makes fp32's forward spill 132 bytes.  Read as volatile, fp32's gradients take
// 86.5 us for 90 at 16384 x 3328 to bf16, bf16's 87.5 for 85.6 and fp32's forward 76.3 for 75.5.)
template <int V, int U, bool GRAD, bool SUBS, class X, class Y>
__global__ void __maxnreg__(registers(U * V, GRAD, V > 1)) block_rows(const Args a)
{
    __shared__ float parts[SUBS ? kMaxSubs : 1][2][16][4];
    __shared__ uint64_t fulls[SUBS ? kMaxSubs : 1][kMaxStages];
    __shared__ int flags[2];
    extern __shared__ __align__(128) unsigned char dynamic[];
    const int sub = SUBS ? threadIdx.y : 0, subs = SUBS ? blockDim.y : 1;
    uint64_t* const full = fulls[sub];
    float (*const part)[16][4] = parts[sub];
    // of several rows' threads each have their own, where the first sums leave their part free
    volatile int* const gave_up = SUBS ? reinterpret_cast<int*>(&part[0][0][2]) : &flags[0];
    using Flag = typename std::conditional<GRAD && sizeof(X) == 4, volatile int, int>::type;
    Flag* const leave = SUBS ? reinterpret_cast<int*>(&part[0][0][3]) : &flags[1];
    unsigned char* const ring = dynamic + (size_t)sub * a.stages * (a.x_slot + a.g_slot);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) tc::bar_init(tc::smem_addr(&full[i]), 1);
        *gave_up = 0, *leave = 0;
        tc::bar_init_fence();
    }
    __syncthreads();
    let_next_begin();
    wait_for_earlier();
    const float inv_n = 1.f / (float)a.width;
    const X* const x = static_cast<const X*>(a.x);
    const Y* const g = static_cast<const Y*>(a.g);
    const auto copy = [&](int64_t row, int stage) {
        unsigned char* const to = ring + stage * (a.x_slot + a.g_slot);
        const uint32_t bar = tc::smem_addr(&full[stage]);
        const Span sx(x + row * a.x_stride, a.width * (int64_t)sizeof(X));
        if constexpr (GRAD) {
            const Span sg(g + row * a.g_stride, a.width * (int64_t)sizeof(Y));
            tc::bar_expect(bar, sx.bytes + sg.bytes);
            tc::copy_bytes(tc::smem_addr(to + a.x_slot), sg.from, sg.bytes, bar);
        } else {
            tc::bar_expect(bar, sx.bytes);
        }
        tc::copy_bytes(tc::smem_addr(to), sx.from, sx.bytes, bar);
    };
    const int64_t mine = (int64_t)blockIdx.x * subs + sub, step = (int64_t)gridDim.x * subs;
    if (threadIdx.x == 0)
        for (int i = 0; i < a.stages; ++i)
            if (mine + i * step < a.rows) copy(mine + i * step, i);
    Piece<V, U, GRAD, true, X, Y> p;
    p.open(a, threadIdx.x, blockDim.x);
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t row = mine; row < a.rows; row += step) {
        tc::bar_wait(tc::smem_addr(&full[stage]), phase, gave_up);
        const unsigned char* const at = ring + stage * (a.x_slot + a.g_slot);
        const uint32_t skip_x = V > 1 ? 0 : (uint32_t)(reinterpret_cast<uintptr_t>(x + row * a.x_stride) & 15);
        const uint32_t skip_g = V > 1 || !GRAD ? 0 : (uint32_t)(reinterpret_cast<uintptr_t>(g + row * a.g_stride) & 15);
        p.row(
            a, reinterpret_cast<const X*>(at + skip_x), reinterpret_cast<const Y*>(at + a.x_slot + skip_g),
            [&] { return a.out && !*leave ? static_cast<typename Piece<V, U, GRAD, true, X, Y>::O*>(a.out) + row * a.width : nullptr; }, true, inv_n,
            [&](auto& s) { block_sums<1, SUBS>(s, part[0], sub); },
            [&](auto& s) {
                if (*gave_up) *leave = 1;
                block_sums<GRAD ? 4 : 2, SUBS>(s, part[1], sub);
            },
            [](bool large) { return large; });
        if (*leave) break;
        // every thread has taken the row for good: the second sums' barrier has been met
        const int64_t next = row + a.stages * step;
        if (threadIdx.x == 0 && next < a.rows) copy(next, stage);
        if (++stage == a.stages) stage = 0, phase ^= 1;
    }
    if (*leave) gave_up_end(threadIdx.x == 0 ? a.status : nullptr);
    if constexpr (GRAD) {
        if (a.dw || a.db) put_sums<Piece<V, U, GRAD, true, X, Y>, V, U>(a, p, reinterpret_cast<float*>(dynamic), subs);
    }
}

// Rows that some lanes, or all of a warp's, can hold: some lanes take one, a warp several, and each warp has its
// own ring of stages, of a.chunk rows each.  No warp waits for another.
template <int V, int U, bool GRAD, class X, class Y>
__global__ void __maxnreg__(registers(U * V, GRAD, V > 1)) warp_rows(const Args a)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ uint64_t full[kWarps][kMaxStages];
    __shared__ int gave_up;
    extern __shared__ __align__(128) unsigned char dynamic[];
    const int thread = threadIdx.y * blockDim.x + threadIdx.x, warp = thread >> 5, lane = thread & 31;
    const int lanes = blockDim.x, at_once = 32 / lanes, sub = lane / lanes;
    if (lane == 0) {
        for (int i = 0; i < a.stages; ++i) tc::bar_init(tc::smem_addr(&full[warp][i]), 1);
        if (warp == 0) gave_up = 0;
        tc::bar_init_fence();
    }
    __syncthreads();
    let_next_begin();
    wait_for_earlier();
    const float inv_n = 1.f / (float)a.width;
    const X* const x = static_cast<const X*>(a.x);
    const Y* const g = static_cast<const Y*>(a.g);
    const int64_t chunks = (a.rows + a.chunk - 1) / a.chunk, step = (int64_t)gridDim.x * kWarps;
    unsigned char* const ring = dynamic + (size_t)warp * a.stages * (a.x_slot + a.g_slot);

    const bool whole = a.x_whole && (!GRAD || a.g_whole);
    const auto copy = [&](int64_t chunk, int stage) {   // the whole warp
        unsigned char* const to = ring + stage * (a.x_slot + a.g_slot);
        const uint32_t bar = tc::smem_addr(&full[warp][stage]);
        const int64_t row = chunk * a.chunk;
        const int have = (int)min((int64_t)a.chunk, a.rows - row);
        if (whole) {
            if (lane == 0) {
                const Span sx(x + row * a.x_stride, (int64_t)have * a.width * sizeof(X)), sg(GRAD ? g + row * a.g_stride : nullptr, GRAD ? (int64_t)have * a.width * sizeof(Y) : 0);
                tc::bar_expect(bar, sx.bytes + sg.bytes);
                tc::copy_bytes(tc::smem_addr(to), sx.from, sx.bytes, bar);
                if (GRAD) tc::copy_bytes(tc::smem_addr(to + a.x_slot), sg.from, sg.bytes, bar);
            }
            return;
        }
        const auto one = [&](const auto* base, int64_t stride, bool whole, int pitch, unsigned char* dst, bool send) {
            const int i = whole ? 0 : lane;
            const Span s(base + (row + i) * stride, (whole ? have : 1) * (int64_t)a.width * sizeof(*base));
            const bool mine = whole ? lane == 0 : lane < have;
            if (send && mine) tc::copy_bytes(tc::smem_addr(dst + i * pitch), s.from, s.bytes, bar);
            return mine ? s.bytes : 0u;
        };
        uint32_t bytes = one(x, a.x_stride, a.x_whole, a.x_pitch, to, false);
        if (GRAD) bytes += one(g, a.g_stride, a.g_whole, a.g_pitch, to + a.x_slot, false);
        bytes = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) tc::bar_expect(bar, bytes);
        __syncwarp();
        one(x, a.x_stride, a.x_whole, a.x_pitch, to, true);
        if (GRAD) one(g, a.g_stride, a.g_whole, a.g_pitch, to + a.x_slot, true);
    };
    // where a stage's first row, or row i by itself, begins beyond a 16-byte boundary
    const auto skip = [](const auto* base, int64_t stride, int64_t row) {
        return V > 1 ? 0 : (int)(reinterpret_cast<uintptr_t>(base + row * stride) & 15);
    };
    const int x_row = a.x_whole ? a.width * (int)sizeof(X) : a.x_pitch, g_row = a.g_whole ? a.width * (int)sizeof(Y) : a.g_pitch;
    using O = typename Piece<V, U, GRAD, false, X, Y>::O;

    const int64_t mine = (int64_t)blockIdx.x * kWarps + warp;
    for (int i = 0; i < a.stages; ++i)
        if (mine + i * step < chunks) copy(mine + i * step, i);
    Piece<V, U, GRAD, false, X, Y> p;
    p.open(a, lane % lanes, lanes);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t chunk = mine; chunk < chunks; chunk += step) {
        if (!(ok = tc::bar_wait_warp(tc::smem_addr(&full[warp][stage]), phase, &gave_up))) break;
        const unsigned char* const at = ring + stage * (a.x_slot + a.g_slot);
        const int64_t first = chunk * a.chunk;
        const int left = (int)min((int64_t)a.chunk, a.rows - first);
        const unsigned char* from_x = at + sub * x_row;
        const unsigned char* from_g = at + a.x_slot + sub * g_row;
        if (a.x_whole) from_x += skip(x, a.x_stride, first);
        if (GRAD && a.g_whole) from_g += skip(g, a.g_stride, first);
        O* out = a.out ? static_cast<O*>(a.out) + (first + sub) * a.width : nullptr;
        for (int i = sub; i < a.chunk; i += at_once) {
            const int sx = a.x_whole ? 0 : skip(x, a.x_stride, first + i), sg = !GRAD || a.g_whole ? 0 : skip(g, a.g_stride, first + i);
            p.row(
                a, reinterpret_cast<const X*>(from_x + sx), reinterpret_cast<const Y*>(from_g + sg), [&] { return out; }, i < left, inv_n,
                [&](auto& s) { lane_sums(s, lanes); }, [&](auto& s) { lane_sums(s, lanes); }, [](bool large) { return __any_sync(0xffffffffu, large) != 0; });
            from_x += at_once * x_row;
            from_g += at_once * g_row;
            if (out) out += at_once * a.width;
        }
        __syncwarp();
        if (chunk + a.stages * step < chunks) copy(chunk + a.stages * step, stage);
        if (++stage == a.stages) stage = 0, phase ^= 1;
    }
    if (!ok) gave_up_end(lane == 0 ? a.status : nullptr);
    if constexpr (GRAD) {
        if (a.dw || a.db) put_sums<Piece<V, U, GRAD, false, X, Y>, V, U>(a, p, reinterpret_cast<float*>(dynamic), blockDim.y);
    }
}

// block_sums of kWideThreads.
template <int N>
__device__ __forceinline__ void wide_sums(float (&s)[N], float (*part)[4])
{
    lane_sums(s, 32);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[threadIdx.x >> 5][i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = part[threadIdx.x & (kWideThreads / 32 - 1)][i];
    lane_sums(s, kWideThreads / 32);
}

// Wider rows: a block takes one, three times over, the later ones from the caches, kWideAhead
// vectors a thread on their way (4000 x 16384 bf16: 231 us with one, by 1024 threads; 9000 x 8193 705, and 412).
constexpr int kWideAhead = 4;

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
        // f(column, its vectors of x and, with_g, of g) for the thread's vectors
        const auto each = [&](bool with_g, auto f) {
            for (int c0 = threadIdx.x * V; c0 < width; c0 += kWideAhead * step) {
                Raw<V, X> v[kWideAhead];
                Raw<V, Y> r[kWideAhead];
#pragma unroll
                for (int i = 0; i < kWideAhead; ++i)
                    if (c0 < width - i * step) {
                        v[i].load_again(x + c0 + i * step);
                        if (with_g) r[i].load_again(g + c0 + i * step);
                    }
#pragma unroll
                for (int i = 0; i < kWideAhead; ++i)
                    if (c0 < width - i * step) f(c0 + i * step, v[i], r[i]);
            }
        };
        Moments mo;
        float along = 0.f, mean_gw = 0.f, scale = 1.f;
        for (bool again = false;; again = true) {
            float s1[1] = {};
            each(false, [&](int, const Raw<V, X>& v, const Raw<V, Y>&) {
#pragma unroll
                for (int q = 0; q < V; ++q) s1[0] += v[q] * scale;
            });
            wide_sums(s1, part[0]);
            const float m = s1[0] * inv_n;
            float s[GRAD ? 4 : 2] = {};
            each(GRAD, [&](int c, const Raw<V, X>& v, const Raw<V, Y>& r) {
                float w[V];
                if (GRAD) params<V>(a.weight, a.param_dtype, c, 1.f, w);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float e = v[q] * scale - m;
                    s[0] += e;
                    s[1] = __fmaf_rn(e, e, s[1]);
                    if constexpr (GRAD) {
                        const float gw = r[q] * w[q];
                        s[2] += gw;
                        s[3] = __fmaf_rn(gw, e, s[3]);
                    }
                }
            });
            wide_sums(s, part[1]);
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
        each(GRAD, [&](int c, const Raw<V, X>& v, const Raw<V, Y>& r) {
            float o[V], w[V], b[V];
            params<V>(a.weight, a.param_dtype, c, 1.f, w);
            if (!GRAD) params<V>(a.bias, a.param_dtype, c, 0.f, b);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float h = mo.h(v[q]);
                if constexpr (GRAD) o[q] = outer * ((r[q] * w[q] - mean_gw) - h * along);
                else o[q] = __fmaf_rn(h, w[q], b[q]);
            }
            if constexpr (GRAD) store_vec<V, X>(static_cast<X*>(a.out) + row * width + c, o);
            else store_vec<V, Y>(static_cast<Y*>(a.out) + row * width + c, o);
        });
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
    constexpr int kAhead = 4;      // rows on their way
    const int64_t step = (int64_t)gridDim.y * kColumnRows;
    if (c < width)
        for (int64_t row0 = (int64_t)blockIdx.y * kColumnRows + threadIdx.y; row0 < a.rows; row0 += kAhead * step) {
            float4 st[kAhead];
            Raw<V, X> v[kAhead];
            Raw<V, Y> g[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int64_t row = row0 + i * step;
                if (row >= a.rows) continue;
                st[i] = a.stats[row];
                v[i].load(static_cast<const X*>(a.x) + row * a.x_stride + c);
                g[i].load(static_cast<const Y*>(a.g) + row * a.g_stride + c);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (row0 + i * step >= a.rows) continue;
                const Moments mo{st[i].x, st[i].y, st[i].z, st[i].w};
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    acc_w[q] = __fmaf_rn(g[i][q], mo.h(v[i][q]), acc_w[q]);
                    acc_b[q] += g[i][q];
                }
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

// Shared memory of its blocks is asked for once a device, as much as there may be.
template <void (*KERNEL)(Args)>
int launch_ring(const Args& a, int blocks, dim3 block, size_t smem, cudaStream_t st)
{
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> sized[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return EMB_ERR_CUDA;
    if (!sized[dev].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes - kOwnBytes) != cudaSuccess) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        sized[dev].store(true, std::memory_order_relaxed);
    }
    return launch_next(KERNEL, blocks, block, smem, st, 1, a);
}

template <class X>
int launch_rows(Args a, int y_dtype, bool vectors, const Shape& s, cudaStream_t st)
{
    return with_type(y_dtype, [&](auto yt) {
        using Y = decltype(yt);
        const auto go = [&](auto v, auto grad) -> int {
            constexpr int V = decltype(v)::value;
            constexpr bool GRAD = decltype(grad)::value;
            if (s.kind == kWideRows) {
                if (int rc = launch_next(wide_rows<V, GRAD, X, Y>, s.blocks, kWideThreads, 0, st, 1, a)) return rc;
                if constexpr (GRAD) {
                    if (a.dw || a.db)
                        return launch_next(wide_columns<V, X, Y>, dim3((a.width + 32 * V - 1) / (32 * V), s.chunks), dim3(32, kColumnRows), 0, st, 1, a);
                }
                return EMB_OK;
            }
            // a stage's rows: whole, or each from its own 16-byte boundary on
            const auto slot = [&](int bytes, int64_t stride, bool& whole, int& pitch) {
                whole = stride == a.width || a.chunk == 1;
                pitch = (a.width * bytes + 15) / 16 * 16 + (V > 1 ? 0 : 16);
                return whole ? ((a.chunk * a.width * bytes + 15) / 16 * 16 + (V > 1 ? 0 : 16)) : a.chunk * pitch;
            };
            const bool warps = s.kind == kWarpRows;
            if (warps) {
                // about kChunkBytes of a stage's rows, so that copies are long; a lane sends a row
                const int at_once = 32 / s.tx, row_bytes = a.width * (int)(sizeof(X) + (GRAD ? sizeof(Y) : 0));
                a.chunk = std::max(at_once, std::min(32, kChunkBytes / row_bytes / at_once * at_once));
            }
            a.x_slot = slot(sizeof(X), a.x_stride, a.x_whole, a.x_pitch);
            if (GRAD) a.g_slot = slot(sizeof(Y), a.g_stride, a.g_whole, a.g_pitch);
            const int stage = (a.x_slot + a.g_slot) * (warps ? kThreads / 32 : s.ty);
            a.stages = std::max(2, std::min(kMaxStages, kRingBytes / s.per_sm / stage));
            size_t smem = (size_t)a.stages * stage;
            if (GRAD && s.ty > 1) smem = std::max(smem, (size_t)s.tx * s.ty * kFew * sizeof(float));
            constexpr int kLong = GRAD || V == 1 ? kFew : kMany;
            const bool few = s.per_thread == kFew;
            const dim3 block(s.tx, s.ty);
            if (warps) return few ? launch_ring<warp_rows<V, kFew / V, GRAD, X, Y>>(a, s.blocks, block, smem, st) : launch_ring<warp_rows<V, kLong / V, GRAD, X, Y>>(a, s.blocks, block, smem, st);
            if constexpr (GRAD) {
                if (s.ty > 1) return launch_ring<block_rows<V, kFew / V, GRAD, true, X, Y>>(a, s.blocks, block, smem, st);
            }
            return few ? launch_ring<block_rows<V, kFew / V, GRAD, false, X, Y>>(a, s.blocks, block, smem, st) : launch_ring<block_rows<V, kLong / V, GRAD, false, X, Y>>(a, s.blocks, block, smem, st);
        };
        constexpr int kVector = sizeof(X) == 2 && sizeof(Y) == 2 ? 8 : 4;   // of fp32 16 bytes, so that lanes' loads meet no bank twice
        const auto with_v = [&](auto grad) {
            return vectors ? go(std::integral_constant<int, kVector>(), grad) : go(std::integral_constant<int, 1>(), grad);
        };
        return a.g ? with_v(std::true_type()) : with_v(std::false_type());
    });
}

#endif  // EMB_NORM_KERNELS

}  // namespace norm
}  // namespace emb

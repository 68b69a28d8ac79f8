// The expert layer's data movement: the stable sort of a batch's assignments
// by expert, the gather of the tokens' rows into expert order, the weighted sum
// back, and the gradients of both.
//
// All of it is bound by memory: each row is read once and written once per
// place it goes to.  16384 tokens, 2 experts each, 3328 wide, fp32 to bf16: sort 9 us,
// gather 61 us (436 MB, 7.1 TB/s with what L2 keeps), its gradient 69 us (6.4 TB/s).
// 32768 tokens, 4 experts each, 2048 wide, bf16: the weighted sum 100 us (6.7 TB/s),
// its gradients 173 us (7.0 TB/s).  The kernels that touch rows therefore walk the
// tokens, not the sorted rows: a token's row (its gradient) is loaded into registers
// once and stored to (combined from) its k places, so the k copies never come from
// memory again.
//
// Rows that are not whole 16-byte vectors go in pairs, or an element a lane, bound by
// the number of loads: 16384 x 2, bf16, gather, its gradient, sum and its gradients
// take 22.5, 24.6, 24.6 and 37 us at 1024 wide, 28.7, 28.7, 28.7 and 43 at 1026, 33,
// 39, 41 and 51 at 1025.  (Vectors from each written row's own 16-byte boundary,
// shifted out of the words around them, took 35, 45, 57 and 200 us.)
#include <algorithm>
#include <condition_variable>
#include <mutex>
#include <type_traits>

#include "dense_internal.cuh"
#include "emb_internal.cuh"
#include "rows.cuh"

namespace emb {
namespace {

constexpr int kMaxDevices = 64;
// The sticky bits, then a place for the bits that a call of emb_dense_status has taken:
// calls of several threads may be under way at once, and each reads its own.
constexpr int kTakers = 64;
__device__ int g_status[1 + kTakers];

std::mutex g_status_mutex;
std::condition_variable g_taker_left;
int* g_status_addr[kMaxDevices] = {};
uint64_t g_takers[kMaxDevices] = {};   // of each device, the places in use

__global__ void take_status(int* status, int place) { status[1 + place] = atomicExch(&status[0], 0); }

// A place of the current device's, waited for while all are in use.
struct Taker {
    int dev = 0, place = -1;
    Taker()
    {
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return;
        std::unique_lock<std::mutex> lock(g_status_mutex);
        g_taker_left.wait(lock, [&] { return g_takers[dev] != ~uint64_t(0); });
        for (place = 0; g_takers[dev] >> place & 1;) ++place;
        g_takers[dev] |= uint64_t(1) << place;
    }
    ~Taker()
    {
        if (place < 0) return;
        {
            std::lock_guard<std::mutex> lock(g_status_mutex);
            g_takers[dev] &= ~(uint64_t(1) << place);
        }
        g_taker_left.notify_all();   // of any device
    }
    Taker(const Taker&) = delete;
    Taker& operator=(const Taker&) = delete;
};

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
// A counting sort in chunks of consecutive assignments, one a block.  With more
// than one chunk, expert_count leaves the chunks' counts in memory, and every
// block of expert_place adds up those before its own instead of waiting for
// them.  Bucket E holds the assignments without an expert, so they too have a
// row, the tail's.  Bound by the latency of its few dependent steps: 4.4 us for one
// block, 3 + 6.4 us for 32768 assignments (in chunks of 8192, eight rounds each:
// 31 us).
constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWarps = kPlaceThreads / 32;
constexpr int kOneChunk = EMB_EXPERT_SORT_ALONE;   // up to so many assignments one block does everything, without expert_count
constexpr int kSms = 152;
constexpr int kMaxChunks = 2 * kSms;           // at most two blocks an SM

template <class ID>
__device__ __forceinline__ int bucket_of(const ID* ids, int64_t a, int E, int* status)
{
    const long long v = (long long)ids[a];
    if (v >= 0 && v < E) return (int)v;
    if (v != -1 && status) atomicOr(status, ERRBIT_KEY_RANGE);
    return E;
}

// counts[bucket][chunk]
template <class ID>
__global__ void __launch_bounds__(kPlaceThreads) expert_count(const ID* __restrict__ ids, int P, int E, int chunk,
                                                              int* __restrict__ counts)
{
    extern __shared__ int cnt[];
    let_next_begin();
    wait_for_earlier();
    for (int e = threadIdx.x; e <= E; e += kPlaceThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * chunk, hi = min((int64_t)P, lo + chunk);
    for (int64_t a = lo + threadIdx.x; a < hi; a += kPlaceThreads) atomicAdd(&cnt[bucket_of(ids, a, E, nullptr)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPlaceThreads) counts[(int64_t)e * gridDim.x + blockIdx.x] = cnt[e];
}

__device__ __forceinline__ int warp_inclusive_scan(int v)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if ((threadIdx.x & 31) >= d) v += u;
    }
    return v;
}

// Exclusive prefix sum of v[0..n) in place, n <= 2 * kPlaceThreads.
__device__ void block_exclusive_scan(int* v, int n, int* warp_sums)
{
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int a = 2 * t < n ? v[2 * t] : 0, b = 2 * t + 1 < n ? v[2 * t + 1] : 0;
    const int s = warp_inclusive_scan(a + b);
    if (lane == 31) warp_sums[w] = s;
    __syncthreads();
    if (w == 0) warp_sums[lane] = warp_inclusive_scan(warp_sums[lane]);
    __syncthreads();
    const int before = s - (a + b) + (w ? warp_sums[w - 1] : 0);
    if (2 * t < n) v[2 * t] = before;
    if (2 * t + 1 < n) v[2 * t + 1] = before + a;
    __syncthreads();
}

// Shared memory: next[E + 1] (the row the next assignment of each bucket gets),
// base[E + 1] (the same at the start of a round), warp_sums[32] and, for each
// bucket, a number a warp: its count, then the earlier warps' sum.
template <class ID>
__global__ void __launch_bounds__(kPlaceThreads) expert_place(const ID* __restrict__ ids, int P, int E, int chunk,
                                                              const int* __restrict__ counts, int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ src, int32_t* __restrict__ pos,
                                                              int* status)
{
    extern __shared__ int smem[];
    int* const next = smem;
    int* const base = next + (E + 1);
    int* const warp_sums = base + (E + 1);
    unsigned short* const of_warp = reinterpret_cast<unsigned short*>(warp_sums + 32);
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int64_t lo = (int64_t)blockIdx.x * chunk, hi = min((int64_t)P, lo + chunk);

    for (int i = t; i < (E + 1) * kPlaceWarps; i += kPlaceThreads) of_warp[i] = 0;
    let_next_begin();
    wait_for_earlier();
    // the first row of every bucket, and of this chunk's part of it
    if (counts) {
        for (int e = w; e <= E; e += kPlaceWarps) {   // a warp adds up a bucket's chunks
            int total = 0, before = 0;
            for (int c = lane; c < (int)gridDim.x; c += 32) {
                const int v = __ldg(&counts[(int64_t)e * gridDim.x + c]);
                if (c < (int)blockIdx.x) before += v;
                total += v;
            }
            total = __reduce_add_sync(0xffffffffu, total);
            before = __reduce_add_sync(0xffffffffu, before);
            if (lane == 0) next[e] = total, base[e] = before;
        }
    } else {
        for (int e = t; e <= E; e += kPlaceThreads) next[e] = 0, base[e] = 0;
        __syncthreads();
        for (int64_t a = lo + t; a < hi; a += kPlaceThreads) atomicAdd(&next[bucket_of(ids, a, E, nullptr)], 1);
    }
    __syncthreads();
    block_exclusive_scan(next, E + 1, warp_sums);
    for (int e = t; e <= E; e += kPlaceThreads) {
        if (blockIdx.x == 0) offsets[e] = next[e];
        next[e] += base[e];
    }

    // kPlaceThreads assignments a round, in order: an assignment's row is its
    // bucket's next one, plus those of earlier warps, plus those of lower lanes
    for (int64_t start = lo; start < hi; start += kPlaceThreads) {
        const int64_t a = start + t;
        const bool has = a < hi;
        const int e = has ? bucket_of(ids, a, E, status) : E + 1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (has && rank == 0) of_warp[e * kPlaceWarps + w] = (unsigned short)__popc(same);
        __syncthreads();
        for (int b = w; b <= E; b += kPlaceWarps) {
            const int mine = of_warp[b * kPlaceWarps + lane];
            const int upto = warp_inclusive_scan(mine);
            if (lane == 31) {
                const int first = next[b];
                base[b] = first;
                next[b] = first + upto;
            }
            of_warp[b * kPlaceWarps + lane] = (unsigned short)(upto - mine);
        }
        __syncthreads();
        if (has) {
            const int row = base[e] + of_warp[e * kPlaceWarps + w] + rank;
            pos[a] = e < E ? row : -1;
            src[row] = e < E ? (int32_t)a : -1;
        }
        if (start + kPlaceThreads < hi) {
            __syncthreads();
            for (int i = t; i < (E + 1) * kPlaceWarps; i += kPlaceThreads) of_warp[i] = 0;
            __syncthreads();
        }
    }
}

size_t place_smem(int E)
{
    return sizeof(int) * (2 * (E + 1) + 32) + sizeof(unsigned short) * (size_t)(E + 1) * kPlaceWarps;
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kUnroll = 4;   // vectors a lane holds at once

// Zero the rows past the last group; warps first, first + step, ... of the
// caller share them.
template <int V, class T>
__device__ __forceinline__ void zero_tail(T* rows, int64_t width, int kept, int P, int64_t first, int64_t step, int lane)
{
    const float zero[V] = {};
    for (int64_t p = kept + first; p < P; p += step)
        for (int64_t c = (int64_t)lane * V; c < width; c += 32 * V) store_vec<V, T>(rows + p * width + c, zero);
}

// LANES lanes take UNROLL vectors each of a token's row.  A row of the grid is the
// row's pieces, its blocks 256 / LANES tokens: nobody divides, which costs as much as
// the loads of a few elements (16384 x 2, 1025 wide, gather: 36.8 us with, 32.7 without).
template <int V, int LANES, int UNROLL>
struct Share {
    static constexpr int kTokens = kRowThreads / LANES, kPiece = LANES * UNROLL * V;
    static constexpr int64_t kMaxRows = 65535;

    static dim3 grid(int64_t tokens, int64_t width)
    {
        return dim3((unsigned)((width + kPiece - 1) / kPiece), (unsigned)std::min((tokens + kTokens - 1) / kTokens, kMaxRows));
    }
    __device__ static int64_t first_token() { return (int64_t)blockIdx.y * kTokens + threadIdx.x / LANES; }
    __device__ static int64_t token_step() { return (int64_t)gridDim.y * kTokens; }
    __device__ static int64_t column() { return (int64_t)blockIdx.x * kPiece + threadIdx.x % LANES * V; }
    __device__ static int64_t warp() { return ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32; }
    __device__ static int64_t warps() { return (int64_t)gridDim.x * gridDim.y * (kRowThreads / 32); }
};

// A token's row is loaded once and stored to each of its k rows (walking the sorted
// rows instead would read it k times).
template <int V, int LANES, class X, class R>
__global__ void __launch_bounds__(kRowThreads) dispatch_rows(emb_expert_plan plan, const X* __restrict__ x,
                                                             int64_t x_stride, int64_t width, R* __restrict__ rows)
{
    using S = Share<V, LANES, kUnroll>;
    const int P = (int)(plan.tokens * plan.k);
    const int64_t c0 = S::column();
    let_next_begin();
    wait_for_earlier();
    for (int64_t token = S::first_token(); token < plan.tokens; token += S::token_step()) {
        Raw<V, X> raw[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (c0 + i * LANES * V < width) raw[i].load(x + token * x_stride + c0 + i * LANES * V);
        float v[kUnroll][V];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) v[i][q] = raw[i][q];
        for (int j = 0; j < plan.k; ++j) {
            const int p = __ldg(&plan.pos[token * plan.k + j]);
            if ((unsigned)p >= (unsigned)P) continue;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (c0 + i * LANES * V < width) store_vec<V, R>(rows + (int64_t)p * width + c0 + i * LANES * V, v[i]);
        }
    }
    zero_tail<V, R>(rows, width, plan_offset(plan.offsets, plan.experts, P), P, S::warp(), S::warps(), threadIdx.x % 32);
}

// out[t] = sum_j w[t, j] rows[pos[t, j]]; without weights, the plain sum (the
// dispatch's gradient).  Bound by memory: ROWS rows' pieces of kSumUnroll vectors
// are on their way at once (one row after another, four vectors each: 105 us where
// this takes 67, and 181 where it takes 90; eight vectors a lane for 2 rows: 77).
// Single elements are more at once, as far as there are registers (16384 x 2, 1025
// wide: 70 us with two and 41 with eight; 32768 x 4, weighted: 145 with two or eight
// and 106 with four).
template <int V, int ROWS, bool WEIGHTED>
constexpr int kSumUnroll = V == 8 ? 2 : ROWS == 4 && WEIGHTED ? 4 : 8 / V;

template <int V, int LANES, class R, class O, bool WEIGHTED, int ROWS>
__global__ void __launch_bounds__(kRowThreads) gather_sum(emb_expert_plan plan, const R* __restrict__ rows,
                                                          int64_t rows_stride, const float* __restrict__ weights,
                                                          int64_t width, O* __restrict__ out)
{
    constexpr int U = kSumUnroll<V, ROWS, WEIGHTED>;
    using S = Share<V, LANES, U>;
    const int P = (int)(plan.tokens * plan.k);
    const int64_t c0 = S::column();
    let_next_begin();
    wait_for_earlier();
    for (int64_t token = S::first_token(); token < plan.tokens; token += S::token_step()) {
        float s[U][V] = {};
        for (int j0 = 0; j0 < plan.k; j0 += ROWS) {
            int p[ROWS];
            float w[ROWS];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                p[j] = j0 + j < plan.k ? __ldg(&plan.pos[token * plan.k + j0 + j]) : -1;
                w[j] = WEIGHTED && j0 + j < plan.k ? __ldg(&weights[token * plan.k + j0 + j]) : 1.f;
            }
            Raw<V, R> v[ROWS][U];
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if ((unsigned)p[j] < (unsigned)P && c0 + i * LANES * V < width)
                        v[j][i].load(rows + p[j] * rows_stride + c0 + i * LANES * V);
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if ((unsigned)p[j] >= (unsigned)P) continue;
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int q = 0; q < V; ++q) s[i][q] = WEIGHTED ? __fmaf_rn(w[j], v[j][i][q], s[i][q]) : s[i][q] + v[j][i][q];
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (c0 + i * LANES * V < width) store_vec<V, O>(out + token * width + c0 + i * LANES * V, s[i]);
    }
}

// Both gradients of the weighted sum in one pass over the rows.  blockDim.x threads
// take a token: its gradient is loaded once for kPart of its experts at a time, and
// each row's dot product is added up over them in a fixed order.
constexpr int kPart = 4;
template <int V>
constexpr int kGradUnroll = 8 / V;   // of a lane's vectors on their way at once (16384 x 2, 1025 wide: 1 92 us, 8 49)

template <int V, class O, class R>
__global__ void __launch_bounds__(kRowThreads) combine_grad(emb_expert_plan plan, const O* __restrict__ grad_out,
                                                            int64_t grad_stride, const R* __restrict__ rows,
                                                            int64_t rows_stride, const float* __restrict__ weights,
                                                            int64_t width, R* __restrict__ grad_rows,
                                                            float* __restrict__ grad_weights)
{
    __shared__ float part[kRowThreads / 32][kPart];
    const int P = (int)(plan.tokens * plan.k), thread = threadIdx.y * blockDim.x + threadIdx.x, lane = thread & 31, warp = thread >> 5;
    const int64_t step = (int64_t)gridDim.x * blockDim.y, next = (int64_t)blockDim.x * V;
    let_next_begin();
    wait_for_earlier();
    // a block's tokens move on together: every thread meets every barrier
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < plan.tokens; t0 += step) {
        const int64_t token = t0 + threadIdx.y;
        const bool has = token < plan.tokens;
        for (int j0 = 0; j0 < plan.k; j0 += kPart) {
            float dot[kPart] = {}, w[kPart] = {};
            int p[kPart];
#pragma unroll
            for (int q = 0; q < kPart; ++q) {
                p[q] = has && j0 + q < plan.k ? __ldg(&plan.pos[token * plan.k + j0 + q]) : -1;
                if ((unsigned)p[q] >= (unsigned)P) p[q] = -1;
                if (p[q] >= 0) w[q] = __ldg(&weights[token * plan.k + j0 + q]);
            }
            const auto step_of = [&](auto many, int64_t c0) {
                constexpr int U = decltype(many)::value;
                Raw<V, O> g[U];
                Raw<V, R> y[U][kPart];
#pragma unroll
                for (int u = 0; u < U; ++u) g[u].load(grad_out + token * grad_stride + c0 + u * next);
#pragma unroll
                for (int q = 0; q < kPart; ++q)
                    if (p[q] >= 0) {
#pragma unroll
                        for (int u = 0; u < U; ++u) y[u][q].load(rows + p[q] * rows_stride + c0 + u * next);
                    }
#pragma unroll
                for (int q = 0; q < kPart; ++q)
                    if (p[q] >= 0) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float d[V];
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                dot[q] = __fmaf_rn(g[u][i], y[u][q][i], dot[q]);
                                d[i] = w[q] * g[u][i];
                            }
                            store_vec<V, R>(grad_rows + (int64_t)p[q] * width + c0 + u * next, d);
                        }
                    }
            };
            if (has) {
                int64_t c = (int64_t)threadIdx.x * V;
                if constexpr (kGradUnroll<V> > 1)
                    for (; c + (kGradUnroll<V> - 1) * next < width; c += kGradUnroll<V> * next) step_of(std::integral_constant<int, kGradUnroll<V>>(), c);
                for (; c < width; c += next) step_of(std::integral_constant<int, 1>(), c);
            }
#pragma unroll
            for (int q = 0; q < kPart; ++q) {
#pragma unroll
                for (int d = 16; d; d >>= 1)
                    if (d < blockDim.x) dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], d);
            }
            float s = 0.f;
            if (blockDim.x > 32) {   // a token's warps meet
#pragma unroll
                for (int q = 0; q < kPart; ++q)
                    if (lane == 0) part[warp][q] = dot[q];
                __syncthreads();
                if (threadIdx.x < kPart)
                    for (int v = 0; v < blockDim.x / 32; ++v) s += part[warp + v][threadIdx.x];
                __syncthreads();
            } else {
#pragma unroll
                for (int q = 0; q < kPart; ++q)
                    if (q == threadIdx.x) s = dot[q];
            }
            if (has && threadIdx.x < kPart && j0 + threadIdx.x < plan.k) grad_weights[token * plan.k + j0 + threadIdx.x] = s;
        }
    }
    const int64_t warps = (int64_t)gridDim.x * (kRowThreads / 32);
    zero_tail<V, R>(grad_rows, width, plan_offset(plan.offsets, plan.experts, P), P,
                    (int64_t)blockIdx.x * (kRowThreads / 32) + warp, warps, lane);
}

template <int N>
using number = std::integral_constant<int, N>;

// f(vector, lanes a token).  Vectors of 8 of at most kShortRow elements are taken by 8
// lanes instead of 32 (32768 x 4: gather 12.3 us for 24.6 at 64 wide, 20.5 for 28.3 at
// 256); pairs (16384 x 2, 1026 wide: gather 28.7 us for 32.8 by elements, its gradient
// 28.7 for 38.9, sum 28.7 for 41.0, its gradients 43.0 for 51.2).
constexpr int64_t kShortRow = 256;

template <class F>
int with_vector(int vector, int64_t width, F f)
{
    if (vector == 8) return width <= kShortRow ? f(number<8>(), number<8>()) : f(number<8>(), number<32>());
    return vector == 2 ? f(number<2>(), number<32>()) : f(number<1>(), number<32>());
}

template <bool WEIGHTED>
int launch_gather_sum(const emb_expert_plan& plan, const void* rows, int rows_dtype, int64_t stride, const float* weights,
                      int64_t width, void* out, int out_dtype, cudaStream_t st)
{
    const int vector = std::min(vector_of(rows, rows_dtype, stride, width), vector_of(out, out_dtype, width, width));
    return with_type(rows_dtype, [&](auto r) {
        return with_type(out_dtype, [&](auto o) {
            using R = decltype(r);
            using O = decltype(o);
            const auto go = [&](auto v, auto lanes, auto at_once) {
                constexpr int V = decltype(v)::value, LANES = decltype(lanes)::value, ROWS = decltype(at_once)::value;
                return launch_next(gather_sum<V, LANES, R, O, WEIGHTED, ROWS>, Share<V, LANES, kSumUnroll<V, ROWS, WEIGHTED>>::grid(plan.tokens, width),
                                   kRowThreads, 0, st, 1, plan, (const R*)rows, stride, weights, width, (O*)out);
            };
            return with_vector(vector, width, [&](auto v, auto lanes) {
                return plan.k <= 1   ? go(v, lanes, number<1>())
                       : plan.k <= 2 ? go(v, lanes, number<2>())
                                     : go(v, lanes, number<4>());
            });
        });
    });
}

}  // namespace

int* dense_status_word()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_status_mutex);
    if (!g_status_addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        g_status_addr[dev] = static_cast<int*>(p);
    }
    return g_status_addr[dev];
}

bool expert_plan_valid(const emb_expert_plan* plan)
{
    if (!plan || plan->tokens < 0 || plan->k < 1 || plan->k > kMaxExpertsPerToken || plan->experts < 1 ||
        plan->experts > kMaxExperts || plan->tokens > INT32_MAX / plan->k)
        return false;
    if (!plan->offsets || !aligned_to(plan->offsets, 4) || !aligned_to(plan->src, 4) || !aligned_to(plan->pos, 4)) return false;
    return plan->tokens == 0 || (plan->src && plan->pos);
}

}  // namespace emb

using namespace emb;

extern "C" int emb_dense_status(void* stream)
{
    int* const word = dense_status_word();
    if (!word) return EMB_ERR_CUDA;
    const Taker taker;
    if (taker.place < 0) return EMB_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int bits = 0;
    take_status<<<1, 1, 0, st>>>(word, taker.place);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(&bits, word + 1 + taker.place, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return EMB_ERR_CUDA;
    return bits & ERRBIT_TIMEOUT ? EMB_ERR_TIMEOUT : bits & ERRBIT_KEY_RANGE ? EMB_ERR_KEY_RANGE : EMB_OK;
}

// Assignments a block of the sort takes: one round, more where that would make
// more than kMaxChunks blocks.
static int sort_chunk(int64_t P)
{
    if (P <= kOneChunk) return kOneChunk;
    const int64_t even = (P + kMaxChunks - 1) / kMaxChunks;
    return (int)((even + kPlaceThreads - 1) / kPlaceThreads * kPlaceThreads);
}
static int sort_chunks(int64_t P) { return (int)((P + sort_chunk(P) - 1) / sort_chunk(P)); }

extern "C" int emb_expert_sort_workspace(int64_t tokens, int32_t k, int32_t experts, size_t* bytes)
{
    if (!bytes || tokens < 0 || k < 1 || k > kMaxExpertsPerToken || experts < 1 || experts > kMaxExperts || tokens > INT32_MAX / k)
        return EMB_ERR_INVALID_ARG;
    const int chunks = sort_chunks(tokens * k);
    *bytes = chunks > 1 ? ((sizeof(int) * (size_t)chunks * (experts + 1) + 255) & ~size_t(255)) : 256;
    return EMB_OK;
}

extern "C" int emb_expert_sort(const void* ids, int32_t id_bytes, const emb_expert_plan* plan, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    size_t need = 0;
    if (!expert_plan_valid(plan) || emb_expert_sort_workspace(plan->tokens, plan->k, plan->experts, &need) != EMB_OK ||
        (id_bytes != 4 && id_bytes != 8) || (!ids && plan->tokens) || !aligned_to(ids, id_bytes) || !workspace ||
        !aligned_to(workspace, 256) || workspace_bytes < need)
        return EMB_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* const word = dense_status_word();
    if (!word) return EMB_ERR_CUDA;
    const int P = (int)(plan->tokens * plan->k), E = plan->experts, chunks = sort_chunks(P), chunk = sort_chunk(P);
    if (P == 0) return cudaMemsetAsync(plan->offsets, 0, sizeof(int32_t) * (E + 1), st) == cudaSuccess ? EMB_OK : EMB_ERR_CUDA;
    int* const counts = chunks > 1 ? static_cast<int*>(workspace) : nullptr;
    const size_t smem = place_smem(E);
    const auto go = [&](auto id) {
        using ID = decltype(id);
        if (smem > 48 * 1024 && cudaFuncSetAttribute(expert_place<ID>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return (int)EMB_ERR_CUDA;
        }
        if (counts) {
            if (int rc = launch_next(expert_count<ID>, chunks, kPlaceThreads, sizeof(int) * (E + 1), st, 1, (const ID*)ids, P, E, chunk, counts)) return rc;
        }
        return launch_next(expert_place<ID>, chunks, kPlaceThreads, smem, st, 1, (const ID*)ids, P, E, chunk, (const int*)counts, plan->offsets, plan->src,
                           plan->pos, word);
    };
    return id_bytes == 4 ? go(int32_t()) : go((long long)0);
}

extern "C" int emb_expert_dispatch(const emb_expert_plan* plan, const void* x, int32_t x_dtype, int64_t x_stride, int64_t width,
                                   void* rows, int32_t rows_dtype, void* stream)
{
    if (!expert_plan_valid(plan) || width < 1 || !rows_valid(x, x_dtype, x_stride, width, plan->tokens) ||
        !rows_valid(rows, rows_dtype, width, width, plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int vector = std::min(vector_of(x, x_dtype, x_stride, width), vector_of(rows, rows_dtype, width, width));
    return with_type(x_dtype, [&](auto xt) {
        return with_type(rows_dtype, [&](auto rt) {
            using X = decltype(xt);
            using R = decltype(rt);
            return with_vector(vector, width, [&](auto v, auto lanes) {
                constexpr int V = decltype(v)::value, LANES = decltype(lanes)::value;
                return launch_next(dispatch_rows<V, LANES, X, R>, Share<V, LANES, kUnroll>::grid(plan->tokens, width), kRowThreads, 0, st, 1, *plan,
                                   (const X*)x, x_stride, width, (R*)rows);
            });
        });
    });
}

extern "C" int emb_expert_dispatch_grad(const emb_expert_plan* plan, const void* grad_rows, int32_t rows_dtype,
                                        int64_t grad_stride, int64_t width, void* grad_x, int32_t x_dtype, void* stream)
{
    if (!expert_plan_valid(plan) || width < 1 || !rows_valid(grad_rows, rows_dtype, grad_stride, width, plan->tokens) ||
        !rows_valid(grad_x, x_dtype, width, width, plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    return launch_gather_sum<false>(*plan, grad_rows, rows_dtype, grad_stride, nullptr, width, grad_x, x_dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int emb_expert_combine(const emb_expert_plan* plan, const void* rows, int32_t rows_dtype, int64_t rows_stride,
                                  const float* weights, int64_t width, void* out, int32_t out_dtype, void* stream)
{
    if (!expert_plan_valid(plan) || width < 1 || !rows_valid(rows, rows_dtype, rows_stride, width, plan->tokens) ||
        !rows_valid(out, out_dtype, width, width, plan->tokens) || !aligned_to(weights, 4) || (!weights && plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    return launch_gather_sum<true>(*plan, rows, rows_dtype, rows_stride, weights, width, out, out_dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int emb_expert_combine_grad(const emb_expert_plan* plan, const void* grad_out, int32_t out_dtype, int64_t grad_stride,
                                       const void* rows, int32_t rows_dtype, int64_t rows_stride, const float* weights,
                                       int64_t width, void* grad_rows, float* grad_weights, void* stream)
{
    if (!expert_plan_valid(plan) || width < 1 || !rows_valid(grad_out, out_dtype, grad_stride, width, plan->tokens) ||
        !rows_valid(rows, rows_dtype, rows_stride, width, plan->tokens) || !rows_valid(grad_rows, rows_dtype, width, width, plan->tokens) ||
        !aligned_to(weights, 4) || !aligned_to(grad_weights, 4) || ((!weights || !grad_weights) && plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int vector = std::min({vector_of(grad_out, out_dtype, grad_stride, width), vector_of(rows, rows_dtype, rows_stride, width),
                                 vector_of(grad_rows, rows_dtype, width, width)});
    // Threads a token: 64 elements each, because the more tokens a block has the less it
    // waits for one, and down to 16 where tokens are too few to fill the GPU.  With 64 and
    // 16, 3328 wide: 16384 x 2 100 and 119 us, 300 x 8 22.5 and 14.3 us.  Less than a warp
    // has 16 (32768 x 4, 64 wide: 28.7 us by 32 threads, 14.3 by 8).
    int tx = vector == 8 ? 8 : 32;
    while (tx < 32 && tx * 16 < width) tx *= 2;
    while (tx >= 32 && tx < kRowThreads && (tx * 64 < width || (tx * 16 < width && plan->tokens * tx * 2 <= kSms * 1024))) tx *= 2;
    const dim3 block(tx, kRowThreads / tx);
    const int64_t b = (plan->tokens + block.y - 1) / block.y;
    const unsigned blocks = (unsigned)(b > (1 << 20) ? (1 << 20) : b);
    return with_type(out_dtype, [&](auto ot) {
        return with_type(rows_dtype, [&](auto rt) {
            using O = decltype(ot);
            using R = decltype(rt);
            return launch_next(vector == 8 ? combine_grad<8, O, R> : vector == 2 ? combine_grad<2, O, R> : combine_grad<1, O, R>, blocks, block, 0, st, 1, *plan, (const O*)grad_out, grad_stride,
                               (const R*)rows, rows_stride, weights, width, (R*)grad_rows, grad_weights);
        });
    });
}

// Dropout with a mask that is computed where it is used, never stored.
//
// Element i of the matrix (row by row, whatever its strides) is kept when its 16 bits
// of Philox4x32 (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011)
// are at least 65536 times the rate.  Counter (i / 8, offset), key the seed: a counter's
// four words are eight elements' bits.  Seven rounds are the fewest with which the
// paper's generator passes its batteries of tests; with 16 bits an element they take
// about five of an element's instructions, and memory stays the bound.
//
// 32768 x 2048 bf16: 40.3 us (6.7 TB/s), with a residual 57.7 (7.0), fp32 with one 113 (7.1); rows 8
// elements apart 63 (6.4).  By elements (rows that are no vectors) 174 us.
#include <algorithm>
#include <cmath>

#include "rows.cuh"

namespace emb {
namespace {

constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u, kW0 = 0x9E3779B9u, kW1 = 0xBB67AE85u;
constexpr int kRounds = 7;
constexpr int kThreads = 256;
constexpr int kGroup = 8;    // elements of a counter

// Bits of a group: element j has the j % 2-th half of word j / 2.
__device__ __forceinline__ uint4 philox(uint64_t group, uint64_t offset, uint64_t seed)
{
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t p0 = (uint64_t)kM0 * c0, p1 = (uint64_t)kM1 * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += kW0, k1 += kW1;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ bool kept(const uint4& bits, int j, uint32_t threshold)
{
    const uint32_t word = j < 2 ? bits.x : j < 4 ? bits.y : j < 6 ? bits.z : bits.w;
    return (j & 1 ? word >> 16 : word & 0xffffu) >= threshold;
}

struct Args {
    const void* x;
    const void* residual;    // nullable
    void* y;
    int64_t x_stride, residual_stride;
    int64_t rows, width;
    const uint64_t* seed_at; // nullable: the seed in device memory
    uint64_t seed, offset;
    uint32_t threshold;
    float scale;
};

// A dropped element is zero whatever it held, an infinity or a NaN too.
template <bool RESIDUAL>
__device__ __forceinline__ float result(bool keep, float x, float residual, float scale)
{
    if (RESIDUAL) return keep ? __fmaf_rn(x, scale, residual) : residual;
    return keep ? x * scale : 0.f;
}

// Groups as vectors of 8: everything is one row, which may end inside a group (FLAT), or
// every row is whole groups.  Bound by memory: a thread has kAhead groups, of as many rows
// where there are rows, on their way before the first is used.
template <class X, class Y, bool RESIDUAL>
constexpr int kAhead = sizeof(X) == 2 && sizeof(Y) == 2 && !RESIDUAL ? 4 : 2;

template <class X, class Y, bool RESIDUAL, bool FLAT>
__global__ void __launch_bounds__(kThreads) drop_groups(const Args a)
{
    constexpr int N = kAhead<X, Y, RESIDUAL>;
    let_next_begin();
    wait_for_earlier();
    const uint64_t seed = a.seed_at ? *a.seed_at : a.seed;
    const int64_t per_row = a.width / kGroup;
    const X* const x = static_cast<const X*>(a.x);
    const Y* const residual = static_cast<const Y*>(a.residual);
    Y* const y = static_cast<Y*>(a.y);
    const int64_t rows_at_once = (int64_t)N * blockDim.y;
    for (int64_t row0 = FLAT ? 0 : blockIdx.y * rows_at_once; row0 < a.rows; row0 += FLAT ? a.rows : gridDim.y * rows_at_once) {
        const auto row_of = [&](int i) { return FLAT ? 0 : row0 + i * (int64_t)blockDim.y + threadIdx.y; };
        const auto group_of = [&](int i) { return FLAT ? (int64_t)blockIdx.x * (kThreads * N) + i * kThreads + threadIdx.x : (int64_t)blockIdx.x * blockDim.x + threadIdx.x; };
        Raw<kGroup, X> v[N];
        Raw<kGroup, Y> r[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (group_of(i) < per_row && (FLAT || row_of(i) < a.rows)) {
                v[i].load(x + row_of(i) * a.x_stride + group_of(i) * kGroup);
                if (RESIDUAL) r[i].load(residual + row_of(i) * a.residual_stride + group_of(i) * kGroup);
            }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t row = row_of(i), c = group_of(i);
            if (!FLAT && row >= a.rows) continue;
            const uint4 bits = philox((uint64_t)(row * per_row + c), a.offset, seed);
            if (c < per_row) {
                float o[kGroup];
#pragma unroll
                for (int j = 0; j < kGroup; ++j) o[j] = result<RESIDUAL>(kept(bits, j, a.threshold), v[i][j], RESIDUAL ? r[i][j] : 0.f, a.scale);
                store_vec<kGroup, Y>(y + row * a.width + c * kGroup, o);
            } else if (FLAT && c == per_row) {   // what is left of the one row
#pragma unroll
                for (int j = 0; j < kGroup; ++j) {
                    const int64_t at = c * kGroup + j;
                    if (at < a.width) y[at] = from_float<Y>(result<RESIDUAL>(kept(bits, j, a.threshold), to_float<X>(x[at]), RESIDUAL ? to_float<Y>(residual[at]) : 0.f, a.scale));
                }
            }
        }
    }
}

// Any sizes, strides and alignments: a warp takes 32 groups, a lane computes one's bits
// and then takes every 32nd element, whose word it gets from the group's lane.
constexpr int kWarpElements = 32 * kGroup;

template <class X, class Y, bool RESIDUAL>
__global__ void __launch_bounds__(kThreads) drop_elements(const Args a)
{
    let_next_begin();
    wait_for_earlier();
    const uint64_t seed = a.seed_at ? *a.seed_at : a.seed;
    const int lane = threadIdx.x & 31;
    const int64_t n = a.rows * a.width, warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t first = ((int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kWarpElements; first < n; first += warps * kWarpElements) {
        const uint4 mine = philox((uint64_t)(first / kGroup + lane), a.offset, seed);
        const int64_t row0 = first / a.width, col0 = first - row0 * a.width;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int from = i * (32 / kGroup) + lane / kGroup, j = lane % kGroup;   // 32 i + lane is group `from`'s element j
            const uint32_t w0 = __shfl_sync(0xffffffffu, mine.x, from), w1 = __shfl_sync(0xffffffffu, mine.y, from);
            const uint32_t w2 = __shfl_sync(0xffffffffu, mine.z, from), w3 = __shfl_sync(0xffffffffu, mine.w, from);
            const uint32_t word = j < 4 ? (j < 2 ? w0 : w1) : (j < 6 ? w2 : w3);
            const bool keep = (j & 1 ? word >> 16 : word & 0xffffu) >= a.threshold;
            const int64_t at = first + i * 32 + lane;
            if (at >= n) continue;
            int64_t row = row0, c = col0 + i * 32 + lane;
            if (a.width >= kWarpElements) {
                if (c >= a.width) c -= a.width, ++row;
            } else {
                const int more = (int)c / (int)a.width;
                row += more, c -= more * a.width;
            }
            const float v = to_float<X>(static_cast<const X*>(a.x)[row * a.x_stride + c]);
            const float r = RESIDUAL ? to_float<Y>(static_cast<const Y*>(a.residual)[row * a.residual_stride + c]) : 0.f;
            static_cast<Y*>(a.y)[at] = from_float<Y>(result<RESIDUAL>(keep, v, r, a.scale));
        }
    }
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" int emb_dropout(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t width, double rate, uint64_t seed,
                           const uint64_t* seed_at, uint64_t offset, const void* residual, int64_t residual_stride, void* y, int32_t y_dtype,
                           void* stream)
{
    if (rows < 0 || width < 1 || width > (int64_t(1) << 40) || rows > (int64_t(1) << 60) / width || !(rate >= 0.0 && rate <= 1.0) ||
        !rows_valid(x, x_dtype, x_stride, width, rows) || !rows_valid(y, y_dtype, width, width, rows) || !aligned_to(seed_at, 8) ||
        (residual && !rows_valid(residual, y_dtype, residual_stride, width, rows)))
        return EMB_ERR_INVALID_ARG;
    if (rows == 0) return EMB_OK;
    Args a = {};
    a.x = x, a.x_stride = x_stride, a.residual = residual, a.residual_stride = residual_stride, a.y = y;
    a.rows = rows, a.width = width, a.seed = seed, a.seed_at = seed_at, a.offset = offset;
    a.threshold = (uint32_t)std::nearbyint(rate * 65536.0);
    a.scale = a.threshold < 65536 ? (float)(1.0 / (1.0 - a.threshold / 65536.0)) : 0.f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // one row of everything, or rows of whole groups, in vectors; else by elements
    const bool flat = (rows == 1 || (x_stride == width && (!residual || residual_stride == width))) && aligned_to(x, 16) && aligned_to(y, 16) &&
                      aligned_to(residual, 16);
    if (flat) a.width = a.x_stride = a.residual_stride = rows * width, a.rows = 1;
    const bool vectors = flat || (vector_of(x, x_dtype, x_stride, width) == 8 && vector_of(y, y_dtype, width, width) == 8 &&
                                  (!residual || vector_of(residual, y_dtype, residual_stride, width) == 8));
    const int64_t groups = (a.width + kGroup - 1) / kGroup;
    return with_type(x_dtype, [&](auto xt) {
        return with_type(y_dtype, [&](auto yt) {
            using X = decltype(xt);
            using Y = decltype(yt);
            const auto go = [&](auto has) -> int {
                constexpr bool RESIDUAL = decltype(has)::value;
                constexpr int N = kAhead<X, Y, RESIDUAL>;
                const auto blocks = [](int64_t n, int64_t each) { return std::min<int64_t>((n + each - 1) / each, INT32_MAX); };
                if (flat) {
                    if (groups > (int64_t)INT32_MAX * kThreads * N) return EMB_ERR_INVALID_ARG;
                    return launch_next(drop_groups<X, Y, RESIDUAL, true>, (unsigned)blocks(groups, kThreads * N), kThreads, 0, st, 1, a);
                }
                if (vectors) {
                    int tx = 1;
                    while (tx < kThreads && tx < groups) tx *= 2;
                    if (groups > (int64_t)INT32_MAX * tx) return EMB_ERR_INVALID_ARG;
                    const dim3 block(tx, kThreads / tx);
                    const dim3 grid((unsigned)blocks(groups, tx), (unsigned)std::min<int64_t>(blocks(a.rows, N * (int64_t)block.y), 65535));
                    return launch_next(drop_groups<X, Y, RESIDUAL, false>, grid, block, 0, st, 1, a);
                }
                return launch_next(drop_elements<X, Y, RESIDUAL>, (unsigned)blocks(rows * width, kThreads * kGroup), kThreads, 0, st, 1, a);
            };
            return residual ? go(std::true_type()) : go(std::false_type());
        });
    });
}

// The whole expert layer for a few tokens, in two kernels.
//
//   hidden[a] = act(up[e] x[t]),  y[a] = down[e] hidden[a],  out[t] = sum_j weights[t, j] y[t k + j]
//
// of assignment a = t k + j to expert e.  Bound by reading the chosen experts' weights,
// once: one request's tokens use each number of them a few times.  So a warp takes
// 16 rows of a weight and reads them straight into registers as the left operand of
// the warp's matrix instruction, 16 bytes a lane; the group's tokens, 8 at a time, are the
// right one.  The order of k within an instruction is free as long as both operands
// agree, so a lane's 8 consecutive elements serve two instructions and nothing passes
// through shared memory.  (The tensor cores' own tiles of 128 rows would leave most SMs
// without one for a single token, and idle otherwise: at 64 tokens an expert the
// products take a tenth of the time the weights do.)
//
// Where there are fewer tiles of 16 rows than warps, the warps of a block share a tile's k
// and add up in shared memory, in order.
//
// Every block makes the groups for itself in shared memory.  The first kernel leaves
// hidden in memory, the second y in fp32; whichever warp finishes the last expert's tile of
// 16 outputs adds up these columns of every token, in the order of j: results repeat bit
// for bit.
#include <algorithm>
#include <type_traits>

#include "emb_internal.cuh"
#include "rows.cuh"

namespace emb {
namespace {

constexpr int kMost = EMB_EXPERT_LAYER_ASSIGNMENTS;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSms = 152, kPerSm = 2;
constexpr int kTile = 16;       // rows of a weight a warp takes
constexpr int kStep = 32;       // k of a lane group's 16 bytes
constexpr int kChunk = 64;      // of a group's assignments at once, at most

struct Args {
    const void* ids;
    int id_bytes, tokens, k, experts;
    const void* x;
    int64_t x_stride;
    const void* up;
    const void* down;
    int in_width, hidden, out_width;
    const float* weights;
    void* out;
    int out_dtype;
    void* hidden_at;         // [assignments][hidden]
    float* y;                // [assignments][out_width]
    int* done;               // of each tile of outputs, the experts
    int* status;
    int share;               // warps of a tile
};

struct Groups {
    int count[kMaxExperts];
    short expert_of[kMost];      // of each assignment, -1: none
    short expert[kMost];         // the experts with assignments, in order
    short first[kMost + 1];      // their first member
    short member[kMost];         // assignments by expert
    int warp_sums[kWarps];
    int active;
};

// The assignments by expert.  Within a group the order is whatever the atomics make it:
// an assignment's results do not depend on its neighbours.
__device__ void make_groups(const Args& a, Groups& g, bool report)
{
    const int t = threadIdx.x, P = a.tokens * a.k;
    for (int e = t; e < a.experts; e += kThreads) g.count[e] = 0;
    __syncthreads();
    for (int i = t; i < P; i += kThreads) {
        const long long id = a.id_bytes == 8 ? __ldg(static_cast<const long long*>(a.ids) + i) : (long long)__ldg(static_cast<const int32_t*>(a.ids) + i);
        const bool has = id >= 0 && id < a.experts;
        if (!has && id != -1 && report) atomicOr(a.status, ERRBIT_KEY_RANGE);
        g.expert_of[i] = has ? (short)id : (short)-1;
        if (has) atomicAdd(&g.count[id], 1);
    }
    __syncthreads();
    // each thread's experts: how many have members, and how many members, in one number
    constexpr int kEach = kMaxExperts / kThreads;
    int mine = 0;
    for (int i = 0; i < kEach; ++i) {
        const int e = t * kEach + i;
        if (e < a.experts && g.count[e]) mine += (1 << 16) + g.count[e];
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, d);
        if ((t & 31) >= d) upto += u;
    }
    if ((t & 31) == 31) g.warp_sums[t >> 5] = upto;
    __syncthreads();
    int before = upto - mine;
    for (int w = 0; w < t >> 5; ++w) before += g.warp_sums[w];
    if (t == kThreads - 1) {
        g.active = (before + mine) >> 16;
        g.first[(before + mine) >> 16] = (short)((before + mine) & 0xffff);
    }
    for (int i = 0; i < kEach; ++i) {
        const int e = t * kEach + i;
        if (e >= a.experts || !g.count[e]) continue;
        g.expert[before >> 16] = (short)e;
        g.first[before >> 16] = (short)(before & 0xffff);
        const int members = g.count[e];
        g.count[e] = before & 0xffff;      // from here on, the next member's place
        before += (1 << 16) + members;
    }
    __syncthreads();
    for (int i = t; i < P; i += kThreads)
        if (g.expert_of[i] >= 0) g.member[atomicAdd(&g.count[g.expert_of[i]], 1)] = (short)i;
    __syncthreads();
}

__device__ __forceinline__ uint4 load_weight(const void* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// 8 elements of a row as the products take them.
template <class T>
__device__ __forceinline__ uint4 load_row(const T* p) { return *reinterpret_cast<const uint4*>(p); }
template <class T>
__device__ __forceinline__ uint4 load_row(const float* p)
{
    const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
    const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    uint4 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) reinterpret_cast<T*>(&r)[i] = from_float<T>(f[i]);
    return r;
}

template <class T>
__device__ __forceinline__ void multiply(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 rows of a weight (rows g and g + 8 of a lane's at w0 and w1, null: none) times NT x 8 rows
// (row(n): the n-th, null: none), over steps [s0, s1) of k.  The weights of the
// next AHEAD steps are on their way while the products of these are made.
template <class T, class X, int NT, class ROW>
__device__ __forceinline__ void products(float (&acc)[NT][4], const T* w0, const T* w1, ROW row, int k, int s0, int s1)
{
    constexpr int AHEAD = NT >= 4 ? 2 : 4;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = (lane & 3) * 8;
    const X* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = row(n * 8 + g);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 a0[2][AHEAD], a1[2][AHEAD];
    const auto fetch = [&](uint4 (&to0)[AHEAD], uint4 (&to1)[AHEAD], int s) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = (s + i) * kStep + c;
            const bool in = s + i < s1 && at < k;
            to0[i] = in && w0 ? load_weight(w0 + at) : zero;
            to1[i] = in && w1 ? load_weight(w1 + at) : zero;
        }
    };
    const auto use = [&](const uint4 (&p)[AHEAD], const uint4 (&q)[AHEAD], int s) {
        constexpr int AT_ONCE = NT >= 4 ? 1 : AHEAD;     // steps whose rows are in registers
#pragma unroll
        for (int i0 = 0; i0 < AHEAD; i0 += AT_ONCE) {
            uint4 b[AT_ONCE][NT];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int at = (s + i0 + i) * kStep + c;
#pragma unroll
                for (int n = 0; n < NT; ++n) b[i][n] = s + i0 + i < s1 && at < k && x[n] ? load_row<T>(x[n] + at) : zero;
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    multiply<T>(acc[n], p[i0 + i].x, q[i0 + i].x, p[i0 + i].y, q[i0 + i].y, b[i][n].x, b[i][n].y);
                    multiply<T>(acc[n], p[i0 + i].z, q[i0 + i].z, p[i0 + i].w, q[i0 + i].w, b[i][n].z, b[i][n].w);
                }
        }
    };
    fetch(a0[0], a1[0], s0);
    for (int s = s0; s < s1; s += 2 * AHEAD) {
        fetch(a0[1], a1[1], s + AHEAD);
        use(a0[0], a1[0], s);
        fetch(a0[0], a1[0], s + 2 * AHEAD);
        use(a0[1], a1[1], s + AHEAD);
    }
}

// f with the smallest of 1, 2, 4 and 8 eights that n fits
template <class F>
__device__ __forceinline__ void with_eights(int n, F f)
{
    if (n <= 8) f(std::integral_constant<int, 1>());
    else if (n <= 16) f(std::integral_constant<int, 2>());
    else if (n <= 32) f(std::integral_constant<int, 4>());
    else f(std::integral_constant<int, 8>());
}

// Walks a weight's tiles.  place(expert, tile, g, &w0, &w1) gives a lane's two rows, row(a) an
// assignment's operand, take(expert's place, tile, n0, rows, acc) has a tile's sums for
// members n0 on of a group, last(tile) comes after a tile's last group.
template <class T, class X, class PLACE, class ROW, class TAKE, class LAST>
__device__ __forceinline__ void walk(const Args& a, const Groups& g, float* shared, int tiles, int k, PLACE place, ROW row, TAKE take, LAST last)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slots = kWarps / a.share, slot = warp / a.share, part = warp % a.share;
    const int steps = (k + kStep - 1) / kStep, each = (steps + a.share - 1) / a.share;
    const int s0 = min(part * each, steps), s1 = min(s0 + each, steps);
    const int total = g.active * tiles, round = (int)gridDim.x * slots;
    // a block's slots go round together: every warp meets every barrier
    for (int item0 = (int)blockIdx.x * slots; item0 < total; item0 += round) {
        const int item = item0 + slot;
        const bool has = item < total;
        const int which = has ? item / tiles : 0, tile = has ? item - which * tiles : 0;
        const int first = g.first[which], rows = has ? g.first[which + 1] - first : 0;
        const T *w0 = nullptr, *w1 = nullptr;
        if (has) place(g.expert[which], tile, lane >> 2, w0, w1);
        // (with shared tiles, the slots of a block go through as many chunks as the longest)
        int longest = rows;
        if (a.share > 1) {
            longest = 0;
            for (int s = 0; s < slots; ++s)
                if (item0 + s < total) {
                    const int w = (item0 + s) / tiles;
                    longest = max(longest, g.first[w + 1] - g.first[w]);
                }
        }
        for (int n0 = 0; n0 < longest; n0 += kChunk) {
            const int have = min(rows - n0, kChunk);
            with_eights(min(longest - n0, kChunk), [&](auto eights) {
                constexpr int NT = decltype(eights)::value;
                float acc[NT][4] = {};
                const auto member_row = [&](int n) -> const X* { return n < have ? row(g.member[first + n0 + n]) : nullptr; };
                if (have > 0) products<T, X, NT>(acc, w0, w1, member_row, k, s0, s1);
                if (a.share > 1) {
                    float* const mine = shared + warp * (NT * 4 * 32) + lane;
#pragma unroll
                    for (int i = 0; i < NT * 4; ++i) mine[i * 32] = acc[i / 4][i % 4];
                    __syncthreads();
                    if (part == 0)
                        for (int p = 1; p < a.share; ++p)
#pragma unroll
                            for (int i = 0; i < NT * 4; ++i) acc[i / 4][i % 4] += mine[(p * NT * 4 + i) * 32];
                    __syncthreads();
                }
                if (part == 0 && have > 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int m = n * 8 + (lane & 3) * 2 + q;
                            if (m < have) take(tile, (int)g.member[first + n0 + m], lane >> 2, acc[n][q], acc[n][2 + q]);
                        }
                }
            });
        }
        if (part == 0 && has) last(tile);
    }
}

template <int ACT>
__device__ __forceinline__ float activate(float v)
{
    if (ACT == EMB_ACT_RELU) return v < 0.f ? 0.f : v;      // a NaN stays one
    if (ACT == EMB_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678f));
    return v / (1.f + expf(-v));
}

constexpr int kShared = kWarps * (kChunk / 8) * 4 * 32;    // floats

// hidden = act(up x), rounded to T, the type the second product takes
template <class T, class X, int ACT>
__global__ void __launch_bounds__(kThreads, kPerSm) layer_up(const Args a)
{
    constexpr bool GATED = ACT == EMB_ACT_SWIGLU;
    __shared__ Groups g;
    __shared__ float shared[kShared];
    wait_for_earlier();
    let_next_begin();      // after the wait: what stood before this kernel is there for the next one's first reads
    make_groups(a, g, blockIdx.x == 0);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < (a.out_width + kTile - 1) / kTile; i += kThreads) a.done[i] = 0;
    const int units = GATED ? kTile / 2 : kTile;       // of hidden a tile has: rows g are gates, g + 8 what they let through
    T* const hidden = static_cast<T*>(a.hidden_at);
    walk<T, X>(
        a, g, shared, (a.hidden + units - 1) / units, a.in_width,
        [&](int expert, int tile, int r, const T*& w0, const T*& w1) {
            const T* const w = static_cast<const T*>(a.up) + (int64_t)expert * (GATED ? 2 : 1) * a.hidden * a.in_width;
            const int m = tile * units + r, m1 = GATED ? a.hidden + m : m + 8;
            if (m < a.hidden) w0 = w + (int64_t)m * a.in_width;
            if (GATED ? m < a.hidden : m1 < a.hidden) w1 = w + (int64_t)m1 * a.in_width;
        },
        [&](int assignment) { return static_cast<const X*>(a.x) + (assignment / a.k) * a.x_stride; },
        [&](int tile, int assignment, int r, float low, float high) {
            T* const to = hidden + (int64_t)assignment * a.hidden + tile * units + r;
            const int left = a.hidden - tile * units - r;
            if constexpr (GATED) {
                if (left > 0) to[0] = from_float<T>(activate<ACT>(low) * high);
            } else {
                if (left > 0) to[0] = from_float<T>(activate<ACT>(low));
                if (left > 8) to[8] = from_float<T>(activate<ACT>(high));
            }
        },
        [](int) {});
}

// y = down hidden, and the tokens' sums
template <class T>
__global__ void __launch_bounds__(kThreads, kPerSm) layer_down(const Args a)
{
    __shared__ Groups g;
    __shared__ float shared[kShared];
    let_next_begin();
    make_groups(a, g, false);      // the ids were there before layer_up's blocks let this kernel begin
    wait_for_earlier();
    const int N = a.out_width;
    const auto store = [&](int token, int col, const float4& v) {
        const int64_t at = (int64_t)token * N + col;
        const float f[4] = {v.x, v.y, v.z, v.w};
        if (a.out_dtype == EMB_F32) store_vec<4, float>(static_cast<float*>(a.out) + at, f);
        else if (a.out_dtype == EMB_F16) store_vec<4, __half>(static_cast<__half*>(a.out) + at, f);
        else store_vec<4, __nv_bfloat16>(static_cast<__nv_bfloat16*>(a.out) + at, f);
    };
    if (!g.active) {
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)a.tokens * (N / 4); i += (int64_t)gridDim.x * kThreads)
            store((int)(i / (N / 4)), (int)(i % (N / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const T* const hidden = static_cast<const T*>(a.hidden_at);
    walk<T, T>(
        a, g, shared, (N + kTile - 1) / kTile, a.hidden,
        [&](int expert, int tile, int r, const T*& w0, const T*& w1) {
            const T* const w = static_cast<const T*>(a.down) + (int64_t)expert * N * a.hidden;
            const int m = tile * kTile + r;
            if (m < N) w0 = w + (int64_t)m * a.hidden;
            if (m + 8 < N) w1 = w + (int64_t)(m + 8) * a.hidden;
        },
        [&](int assignment) { return hidden + (int64_t)assignment * a.hidden; },
        [&](int tile, int assignment, int r, float low, float high) {
            float* const to = a.y + (int64_t)assignment * N + tile * kTile + r;
            to[0] = low;
            if (tile * kTile + r + 8 < N) to[8] = high;
        },
        [&](int tile) {
            const int lane = threadIdx.x & 31;
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0) before = atomicAdd(&a.done[tile], 1);
            before = __shfl_sync(0xffffffffu, before, 0);
            if (before != g.active - 1) return;
            __threadfence();
            const int col = tile * kTile + (lane & 3) * 4;
            if (col >= N) return;
            for (int t = lane >> 2; t < a.tokens; t += 8) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int j = 0; j < a.k; ++j) {
                    const int p = t * a.k + j;
                    if (g.expert_of[p] < 0) continue;
                    const float w = __ldg(&a.weights[p]);
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.y + (int64_t)p * N + col));
                    s.x = __fmaf_rn(w, v.x, s.x), s.y = __fmaf_rn(w, v.y, s.y), s.z = __fmaf_rn(w, v.z, s.z), s.w = __fmaf_rn(w, v.w, s.w);
                }
                store(t, col, s);
            }
        });
}

size_t rounded(size_t n) { return (n + 255) & ~size_t(255); }

struct Room {
    size_t hidden, y, done;
    Room(int64_t assignments, int64_t hidden_width, int64_t out_width)
        : hidden(rounded((size_t)assignments * hidden_width * 2)), y(rounded((size_t)assignments * out_width * sizeof(float))),
          done(rounded((size_t)(out_width + kTile - 1) / kTile * sizeof(int)))
    {
    }
};

bool widths_valid(int64_t w) { return w >= 8 && w % 8 == 0 && w <= (1 << 24); }

bool sizes_valid(int64_t tokens, int32_t k, int64_t hidden, int64_t out_width)
{
    return tokens >= 0 && k >= 1 && k <= kMaxExpertsPerToken && tokens <= kMost / k && widths_valid(hidden) && widths_valid(out_width);
}

// Warps that share a tile's k: as many as keep eight warps of every SM busy, but four
// steps of k for each.
int sharing(int64_t tiles, int64_t k)
{
    int share = 1;
    while (share < kWarps && tiles * share < kSms * 8 && (k / kStep) / (share * 2) >= 4) share *= 2;
    return share;
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" int emb_expert_layer_workspace(int64_t tokens, int32_t k, int64_t hidden, int64_t out_width, size_t* bytes)
{
    if (!bytes || !sizes_valid(tokens, k, hidden, out_width)) return EMB_ERR_INVALID_ARG;
    const Room r(tokens * k, hidden, out_width);
    *bytes = r.hidden + r.y + r.done;
    return EMB_OK;
}

extern "C" int emb_expert_layer(const void* ids, int32_t id_bytes, int64_t tokens, int32_t k, int32_t experts, const void* x, int32_t x_dtype,
                                int64_t x_stride, int64_t in_width, const void* up, const void* down, int32_t dtype, int64_t hidden,
                                int64_t out_width, int32_t activation, const float* weights, void* out, int32_t out_dtype, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    size_t need = 0;
    if (emb_expert_layer_workspace(tokens, k, hidden, out_width, &need) != EMB_OK || !widths_valid(in_width) || experts < 1 ||
        experts > kMaxExperts || (id_bytes != 4 && id_bytes != 8) || (dtype != EMB_F16 && dtype != EMB_BF16) ||
        (x_dtype != dtype && x_dtype != EMB_F32) || !dtype_valid(out_dtype) || activation < EMB_ACT_RELU || activation > EMB_ACT_SWIGLU ||
        !workspace || !aligned_to(workspace, 256) || workspace_bytes < need)
        return EMB_ERR_INVALID_ARG;
    if (tokens == 0) return EMB_OK;
    if (!ids || !aligned_to(ids, id_bytes) || !x || !aligned_to(x, 16) || x_stride < in_width || x_stride * (int64_t)dtype_bytes(x_dtype) % 16 ||
        !up || !aligned_to(up, 16) || !down || !aligned_to(down, 16) || !weights || !aligned_to(weights, 4) || !out || !aligned_to(out, 16))
        return EMB_ERR_INVALID_ARG;
    Args a = {};
    a.ids = ids, a.id_bytes = id_bytes, a.tokens = (int)tokens, a.k = k, a.experts = experts;
    a.x = x, a.x_stride = x_stride, a.up = up, a.down = down;
    a.in_width = (int)in_width, a.hidden = (int)hidden, a.out_width = (int)out_width;
    a.weights = weights, a.out = out, a.out_dtype = out_dtype;
    const Room room(tokens * k, hidden, out_width);
    unsigned char* const at = static_cast<unsigned char*>(workspace);
    a.hidden_at = at, a.y = reinterpret_cast<float*>(at + room.hidden), a.done = reinterpret_cast<int*>(at + room.hidden + room.y);
    if (!(a.status = dense_status_word())) return EMB_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t groups = std::min<int64_t>(tokens * k, experts);     // at most
    const auto blocks = [](int64_t tiles, int share) { return (unsigned)std::min<int64_t>((tiles * share + kWarps - 1) / kWarps, kSms * kPerSm); };
    const auto go = [&](auto t) -> int {
        using T = decltype(t);
        const int units = activation == EMB_ACT_SWIGLU ? kTile / 2 : kTile;
        const int64_t up_tiles = groups * ((hidden + units - 1) / units), down_tiles = groups * ((out_width + kTile - 1) / kTile);
        const auto first = [&](auto xt) -> int {
            using X = decltype(xt);
            a.share = sharing(up_tiles, in_width);
            const auto kernel = activation == EMB_ACT_RELU   ? layer_up<T, X, EMB_ACT_RELU>
                                : activation == EMB_ACT_SILU ? layer_up<T, X, EMB_ACT_SILU>
                                : activation == EMB_ACT_GELU ? layer_up<T, X, EMB_ACT_GELU>
                                                             : layer_up<T, X, EMB_ACT_SWIGLU>;
            return launch_next(kernel, blocks(up_tiles, a.share), kThreads, 0, st, 1, a);
        };
        if (int rc = x_dtype == EMB_F32 ? first(float()) : first(T())) return rc;
        a.share = sharing(down_tiles, hidden);
        return launch_next(layer_down<T>, blocks(down_tiles, a.share), kThreads, 0, st, 1, a);
    };
    return dtype == EMB_F16 ? go(__half()) : go(__nv_bfloat16());
}

// The expert layer for a few tokens: what its kernels share (sm_103a).
#pragma once

#include <algorithm>
#include <type_traits>

#include "emb_internal.cuh"
#include "rows.cuh"

namespace emb {
namespace few {

constexpr int kMost = EMB_EXPERT_LAYER_ASSIGNMENTS;
constexpr int kSms = 152;
constexpr int kTile = 16;       // rows of a weight a warp takes, outputs that share a token's count

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
    void* rows;              // [assignments, by group][in_width], of the tiles
    void* hidden_at;         // [assignments, by group][hidden]
    float* y;                // [assignments][out_width]
    int* done;               // [tiles of outputs][tokens]: a token's assignments that are done (null: layer_sum adds up)
    int* status;
    int act;
    int share;               // warps of a tile
};

struct Groups {
    short expert_of[kMost];      // of each assignment, -1: none
    unsigned char experts[kMost];   // of each token, how many
    short expert[kMost];         // the experts with assignments, in order
    short first[kMost + 1];      // their first member
    short member[kMost];         // assignments by expert, each expert's in order
    int warp_sums[8];
    int active;
};

// The expert of an assignment, -1: none.
__device__ __forceinline__ int id_of(const Args& a, int i, bool report)
{
    const long long id = a.id_bytes == 8 ? static_cast<const long long*>(a.ids)[i] : (long long)static_cast<const int32_t*>(a.ids)[i];
    if (id >= 0 && id < a.experts) return (int)id;
    if (id != -1 && report) atomicOr(a.status, ERRBIT_KEY_RANGE);
    return -1;
}

// The assignments by expert, a stable sort, by the block's first 8 warps; the whole
// block meets.  `counts`: kCountBytes of shared memory, 16-byte aligned, free afterwards.
constexpr int kCountBytes = kMaxExperts * (kMost / 32);
__device__ __forceinline__ void make_groups(const Args& a, Groups& g, unsigned char* counts, bool report)
{
    constexpr int kRounds = kMost / 32, kThreads = 256;
    static_assert(kRounds == 16, "an expert's counts are one vector");
    const int t = threadIdx.x, lane = t & 31, P = a.tokens * a.k;
    const unsigned below = (1u << lane) - 1;
    if (P <= 32) {      // one warp, without counting (1 token: 1 us less of each kernel)
        if (t < 32) {
            const int id = t < P ? id_of(a, t, report) : -1;
            const unsigned all = __ballot_sync(0xffffffffu, id >= 0), same = __match_any_sync(0xffffffffu, id) & all;
            const bool leads = id >= 0 && !(same & below);
            const unsigned leaders = __ballot_sync(0xffffffffu, leads);
            int before = 0, place = 0;      // members of smaller experts' groups, and these groups
            for (unsigned l = leaders; l; l &= l - 1) {
                const int from = __ffs(l) - 1, members = __popc(__shfl_sync(0xffffffffu, same, from)), other = __shfl_sync(0xffffffffu, id, from);
                if (other < id) before += members, ++place;
            }
            if (t < P) g.expert_of[t] = (short)id;
            if (leads) {
                g.expert[place] = (short)id;
                g.first[place] = (short)before;
            }
            if (id >= 0) g.member[before + __popc(same & below)] = (short)t;
            if (t == 0) {
                g.active = __popc(leaders);
                g.first[__popc(leaders)] = (short)__popc(all);
            }
            if (t < a.tokens) g.experts[t] = (unsigned char)__popc(all >> (t * a.k) & (a.k < 32 ? (1u << a.k) - 1 : ~0u));
        }
        __syncthreads();
        return;
    }
    // counts[expert][round of 32 assignments], then the members in earlier rounds
    uint4* const rounds = reinterpret_cast<uint4*>(counts);
    if (t < kThreads)
        for (int e = t; e < a.experts; e += kThreads) rounds[e] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int id[kMost / kThreads], rank[kMost / kThreads];
    if (t < kThreads)
#pragma unroll
        for (int i = 0; i < kMost / kThreads; ++i) {
            const int at = i * kThreads + t;
            id[i] = at < P ? id_of(a, at, report) : -1;
            const unsigned same = __match_any_sync(0xffffffffu, id[i]);
            rank[i] = __popc(same & below);
            if (at < P) g.expert_of[at] = (short)id[i];
            if (id[i] >= 0 && rank[i] == 0) counts[id[i] * kRounds + at / 32] = (unsigned char)__popc(same);
        }
    __syncthreads();
    // each thread's experts: how many have members, and how many members, in one number
    constexpr int kEach = kMaxExperts / kThreads;
    int mine = 0, total[kEach];
    if (t < kThreads)
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            total[i] = 0;
            const int e = t * kEach + i;
            if (e < a.experts) {
                const uint4 c = rounds[e];
                total[i] = (int)(__dp4a(c.x, 0x01010101u, 0u) + __dp4a(c.y, 0x01010101u, 0u) + __dp4a(c.z, 0x01010101u, 0u) + __dp4a(c.w, 0x01010101u, 0u));
            }
            if (total[i]) mine += (1 << 16) + total[i];
        }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += u;
    }
    if (t < kThreads && lane == 31) g.warp_sums[t >> 5] = upto;
    __syncthreads();
    int start[kMost / kThreads];
    if (t < kThreads) {
        int before = upto - mine;
        for (int w = 0; w < t >> 5; ++w) before += g.warp_sums[w];
        if (t == kThreads - 1) {
            g.active = (before + mine) >> 16;
            g.first[(before + mine) >> 16] = (short)((before + mine) & 0xffff);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (!total[i]) continue;
            const int e = t * kEach + i;
            g.expert[before >> 16] = (short)e;
            g.first[before >> 16] = (short)(before & 0xffff);
            before += (1 << 16) + total[i];
        }
    }
    __syncthreads();
    // an assignment's place: its group's first, those of earlier rounds, those of lower lanes
    if (t < kThreads) {
#pragma unroll
        for (int i = 0; i < kMost / kThreads; ++i) {
            if (id[i] < 0) continue;
            const int at = i * kThreads + t;
            int lo = 0, hi = g.active - 1;       // the group
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (g.expert[mid] < id[i]) lo = mid + 1; else hi = mid;
            }
            start[i] = g.first[lo] + rank[i];
            for (int r = 0; r < at / 32; ++r) start[i] += counts[id[i] * kRounds + r];
            g.member[start[i]] = (short)at;
        }
        for (int token = t; token < a.tokens; token += kThreads) {
            int n = 0;
            for (int j = 0; j < a.k; ++j) n += g.expert_of[token * a.k + j] >= 0;
            g.experts[token] = (unsigned char)n;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float activate(int act, float v)
{
    if (act == EMB_ACT_RELU) return v < 0.f ? 0.f : v;      // a NaN stays one
    // 1 + erf(v / sqrt 2), which loses its digits where erf comes near -1
    if (act == EMB_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678f);
    return v / (1.f + expf(-v));
}

// Four columns of a token's output.
__device__ __forceinline__ void store_out(const Args& a, int token, int col, const float4& v)
{
    const int64_t at = (int64_t)token * a.out_width + col;
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (a.out_dtype == EMB_F32) store_vec<4, float>(static_cast<float*>(a.out) + at, f);
    else if (a.out_dtype == EMB_F16) store_vec<4, __half>(static_cast<__half*>(a.out) + at, f);
    else store_vec<4, __nv_bfloat16>(static_cast<__nv_bfloat16*>(a.out) + at, f);
}

// Four columns of a token: the weighted sum of its rows of y, in the order of j.
// has(p): whether assignment p has one.
template <class HAS>
__device__ __forceinline__ void sum_token(const Args& a, HAS has, int token, int col)
{
    constexpr int kAhead = 8;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
        float4 v[kAhead];
        float w[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int p = token * a.k + j0 + j;
            w[j] = 0.f;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + j < a.k && has(p)) {
                w[j] = __ldg(&a.weights[p]);
                v[j] = __ldcg(reinterpret_cast<const float4*>(a.y + (int64_t)p * a.out_width + col));
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            s.x = __fmaf_rn(w[j], v[j].x, s.x), s.y = __fmaf_rn(w[j], v[j].y, s.y), s.z = __fmaf_rn(w[j], v[j].z, s.z), s.w = __fmaf_rn(w[j], v[j].w, s.w);
    }
    store_out(a, token, col, s);
}

// Tokens without an expert: zeros.  (The first kernel's blocks share them out; nothing
// of the second touches them.)
__device__ __forceinline__ void store_nothing(const Args& a, const Groups& g)
{
    const int quads = a.out_width / 4;
    for (int t = blockIdx.x; t < a.tokens; t += gridDim.x)
        if (!g.experts[t])
            for (int c = threadIdx.x; c < quads; c += blockDim.x) store_out(a, t, c * 4, make_float4(0.f, 0.f, 0.f, 0.f));
}

// No assignment of any tile is done.
__device__ __forceinline__ void clear_done(const Args& a)
{
    const int n = (a.out_width + kTile - 1) / kTile * a.tokens;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) a.done[i] = 0;
}

// few_tiles.cu: hidden and y with the weights' tiles on the tensor cores.  dtype of the weights.
int launch_tiles(const Args& a, int x_dtype, int dtype, cudaStream_t st);

}  // namespace few
}  // namespace emb

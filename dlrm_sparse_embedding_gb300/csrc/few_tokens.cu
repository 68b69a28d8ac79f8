// The whole expert layer for a few tokens.
//
//   hidden[a] = act(up[e] x[t]),  y[a] = down[e] hidden[a],  out[t] = sum_j weights[t, j] y[t k + j]
//
// of assignment a = t k + j to expert e.  Bound by reading the chosen experts' weights, once for
// each kChunk of an expert's assignments: one request's tokens use each number of them a few times.  So a warp takes
// 16 rows of a weight and reads them straight into registers as the left operand of
// the warp's matrix instruction, 16 bytes a lane; the group's tokens, 8 at a time, are the
// right one.  The order of k within an instruction is free as long as both operands
// agree, so a lane's 8 consecutive elements serve two instructions and nothing passes
// through shared memory.  (Tiles of 128 rows on the tensor cores leave most SMs without one
// for a single token; many_weights says from where on they are faster, few_tiles.cu has them.)
//
// Where there are fewer tiles of 16 rows than warps, the warps of a block share a tile's k
// and add up in shared memory, in order.
//
// Two kernels, and up to kSumInDown assignments no more: whoever finishes a tile of outputs of a
// token's last assignment adds up these columns of the token.  A third one does beyond.
// Either adds in the order of j, so results repeat bit for bit.  Every block makes the groups
// for itself in shared memory.
//
// One token, 2 of 16 experts, 3328 -> 1024 -> 1024, fp32 tokens, bf16: 14 us (18 MB; 7 us are what the two kernels
// take with 64 wide weights); 8 tokens 28 us (80 MB, 2.9 TB/s): layer_down's weights come from DRAM only when
// layer_up is done, but for the first steps.  256 x 2 of 4, 2048 wide, each weight read twice: 89 us (tiles 48).
// One kernel holds the products of 8, 16, 32 and 64 of a group, and the two blocks an SM leave it 128 registers: 36 to 140
// bytes a thread spill.  Measured and not kept: twice the weights on their way,
// in one block an SM (14.0 us for 14.3, 26.0 for 25.9); rows ahead with the weights (13.7 and 27.1).
#include <cmath>

#include "few_tokens.cuh"

namespace emb {
namespace {

using namespace few;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPerSm = 2;
// Assignments up to which layer_down adds up the tokens itself: a third launch costs 2 us, the last warps' sums more
// (64 x 8 of 8 in 64 columns: 29 us, and 16 with a third kernel).
constexpr int kSumInDown = 32;
constexpr int kStep = 32;       // k of a lane group's 16 bytes
constexpr int kChunk = 64;      // of a group's assignments at once, at most
constexpr int kShared = kWarps * (kChunk / 8) * 4 * 32;    // floats that warps add up through
static_assert(kShared * (int)sizeof(float) >= kCountBytes, "the groups are made there");

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
// next AHEAD steps are on their way while the products of these are made; ready() comes
// between the first of them and the first row.
template <class T, class X, int NT, class ROW, class READY>
__device__ __forceinline__ void products(float (&acc)[NT][4], const T* w0, const T* w1, ROW row, int k, int s0, int s1, READY ready)
{
    constexpr int AHEAD = NT >= 4 ? 2 : 4;
    constexpr int AT_ONCE = NT >= 4 ? 1 : AHEAD;     // steps whose rows are in registers
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
    ready();
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

// Walks a weight's tiles.  place(expert, tile, i) gives a lane's row, i 0 or 1, row(a) an
// assignment's operand, take(tile, a, low, high) has an assignment's sums for the two, last(tile,
// first, rows) comes after a group's tile.
template <class T, class X, class READY, class PLACE, class ROW, class TAKE, class LAST>
__device__ __forceinline__ void walk(const Args& a, const Groups& g, float* shared, int tiles, int k, READY ready, PLACE place, ROW row, TAKE take,
                                     LAST last)
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
        const T* const w0 = has ? place(g.expert[which], tile, 0) : nullptr;
        const T* const w1 = has ? place(g.expert[which], tile, 1) : nullptr;
        // (with shared tiles, the slots of a block go through as many chunks as the longest)
        int longest = rows;
        if (a.share > 1) {
            longest = 0;
            for (int s = 0; s < slots; ++s)
                if (item0 + s < total) {
                    const int o = (item0 + s) / tiles;
                    longest = max(longest, g.first[o + 1] - g.first[o]);
                }
        }
        for (int n0 = 0; n0 < longest; n0 += kChunk) {
            const int have = min(rows - n0, kChunk);
            with_eights(min(longest - n0, kChunk), [&](auto eights) {
                constexpr int NT = decltype(eights)::value;
                float acc[NT][4] = {};
                const auto member_row = [&](int n) -> const X* { return n < have ? row(g.member[first + n0 + n]) : nullptr; };
                if (have > 0) products<T, X, NT>(acc, w0, w1, member_row, k, s0, s1, ready);
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
                            const int r = n * 8 + (lane & 3) * 2 + q;
                            if (r < have) take(tile, (int)g.member[first + n0 + r], acc[n][q], acc[n][2 + q]);
                        }
                }
            });
        }
        if (part == 0 && has) last(tile, first, rows);
    }
}

// hidden = act(up x), rounded to T: the second product's operands are 16-bit numbers, as in expert_linear.  Of bf16's
// output 2.3e-3 of its size is off 64 bits, 1.7e-3 where hidden stays fp32 (fp16 2.9e-4 and 2.1e-4): the output's own
// rounding is the larger part.  Nothing else of the call is held in fewer bits than fp32.
template <class T, class X, bool GATED>
__global__ void __launch_bounds__(kThreads, kPerSm) layer_up(const Args a)
{
    __shared__ Groups g;
    __shared__ __align__(16) float shared[kShared];
    wait_for_earlier();
    let_next_begin();      // after the wait: what stood before this kernel is there for the next one's first reads
    make_groups(a, g, reinterpret_cast<unsigned char*>(shared), blockIdx.x == 0);
    if (a.done) {
        clear_done(a);
        store_nothing(a, g);
    }
    constexpr int kUnits = GATED ? kTile / 2 : kTile;       // of hidden a tile has: 8 gates and what they let through, or 16 rows
    const int r = (threadIdx.x & 31) >> 2;
    T* const hidden = static_cast<T*>(a.hidden_at);
    walk<T, X>(
        a, g, shared, (a.hidden + kUnits - 1) / kUnits, a.in_width, [] {},
        [&](int expert, int tile, int i) -> const T* {
            const int m = tile * kUnits + r + (GATED ? 0 : i * 8);
            if (m >= a.hidden) return nullptr;
            return static_cast<const T*>(a.up) + ((int64_t)expert * (GATED ? 2 : 1) * a.hidden + (GATED ? i * a.hidden : 0) + m) * a.in_width;
        },
        [&](int assignment) { return static_cast<const X*>(a.x) + (assignment / a.k) * a.x_stride; },
        [&](int tile, int assignment, float low, float high) {
            const int unit = tile * kUnits + r, left = a.hidden - unit;
            T* const to = hidden + (int64_t)assignment * a.hidden + unit;
            if constexpr (GATED) {
                if (left > 0) to[0] = from_float<T>(activate(EMB_ACT_SILU, low) * high);
            } else {
                if (left > 0) to[0] = from_float<T>(activate(a.act, low));
                if (left > 8) to[8] = from_float<T>(activate(a.act, high));
            }
        },
        [](int, int, int) {});
}

// Where the n-th bit of a mask is (somewhere, if it has no more than n).
__device__ __forceinline__ int nth_bit(unsigned mask, int n)
{
    int at = 0;
#pragma unroll
    for (int w = 16; w; w >>= 1) {
        const int c = __popc(mask >> at & ((1u << w) - 1));
        if (n >= c) n -= c, at += w;
    }
    return at & 31;
}

// y = down hidden, and the tokens' sums
template <class T>
__global__ void __launch_bounds__(kThreads, kPerSm) layer_down(const Args a)
{
    __shared__ Groups g;
    __shared__ __align__(16) float shared[kShared];
    let_next_begin();
    make_groups(a, g, reinterpret_cast<unsigned char*>(shared), false);      // the ids, and the first weights, were there before layer_up's blocks let this kernel begin
    const int N = a.out_width, lane = threadIdx.x & 31, r = lane >> 2;
    const T* const hidden = static_cast<const T*>(a.hidden_at);
    walk<T, T>(
        a, g, shared, (N + kTile - 1) / kTile, a.hidden, [] { wait_for_earlier(); },
        [&](int expert, int tile, int i) -> const T* {
            const int m = tile * kTile + i * 8 + r;
            return m < N ? static_cast<const T*>(a.down) + ((int64_t)expert * N + m) * a.hidden : nullptr;
        },
        [&](int assignment) { return hidden + (int64_t)assignment * a.hidden; },
        [&](int tile, int assignment, float low, float high) {
            const int col = tile * kTile + r;
            float* const to = a.y + (int64_t)assignment * N + col;
            to[0] = low;
            if (col + 8 < N) to[8] = high;
        },
        [&](int tile, int first, int rows) {
            if (!a.done) return;
            // whose last assignment this was is added up, eight tokens at a time by four lanes each
            __threadfence();
            __syncwarp();
            int token = 0;
            bool whole = false;
            if (lane < rows) {
                token = g.member[first + lane] / a.k;
                whole = atomicAdd(&a.done[tile * a.tokens + token], 1) == g.experts[token] - 1;
            }
            const unsigned all = __ballot_sync(0xffffffffu, whole);
            if (!all) return;
            __threadfence();
            const int col = tile * kTile + (lane & 3) * 4;
            for (int i = 0; i < __popc(all); i += 8) {
                const int t = __shfl_sync(0xffffffffu, token, nth_bit(all, i + (lane >> 2)));
                if (i + (lane >> 2) < __popc(all) && col < N) sum_token(a, [&](int p) { return g.expert_of[p] >= 0; }, t, col);
            }
        });
    wait_for_earlier();      // a block without a tile, too: what follows takes this kernel's end for both
}

// The tokens' sums: a thread has four columns of one.
__global__ void __launch_bounds__(kThreads) layer_sum(const Args a)
{
    let_next_begin();
    wait_for_earlier();
    const int col = (blockIdx.x * kThreads + threadIdx.x) * 4;
    if (col < a.out_width) sum_token(a, [&](int p) { return id_of(a, p, false) >= 0; }, blockIdx.y, col);
}

size_t rounded(size_t n) { return (n + 255) & ~size_t(255); }

struct Room {
    size_t rows, hidden, y, done;
    Room(int64_t tokens, int64_t assignments, int64_t in_width, int64_t hidden_width, int64_t out_width)
        : rows(rounded((size_t)assignments * in_width * 2)), hidden(rounded((size_t)assignments * hidden_width * 2)),
          y(rounded((size_t)assignments * out_width * sizeof(float))),
          done(rounded((size_t)(out_width + kTile - 1) / kTile * std::min<int64_t>(tokens, kSumInDown) * sizeof(int)))
    {
    }
    size_t all() const { return rows + hidden + y + done; }
};

bool widths_valid(int64_t w) { return w >= 8 && w % 8 == 0 && w <= (1 << 24); }

bool sizes_valid(int64_t tokens, int32_t k, int64_t in_width, int64_t hidden, int64_t out_width)
{
    return widths_valid(in_width) && tokens >= 0 && k >= 1 && k <= kMaxExpertsPerToken && tokens <= kMost / k && widths_valid(hidden) && widths_valid(out_width);
}

// Whether tiles on the tensor cores are faster, by megabytes of weights of the experts that tokens which choose any
// k of them alike would choose.  Tiles save 10 ns a megabyte and 7.5 more for each assignment of
// a group, whose rows the warps here load again for every 16 rows of a weight, and 50 ns a megabyte of `up`
// where they are fp32, converted each time.  They cost what their kernels take to begin and end
// and a ring's way through k: 2 ns an element of a token's row and of hidden.
// Both ways were measured on 740 shapes, most within 12 us of each other: the rule takes the faster one, or
// one within 3 %, on 690 of them, the slowest choice is 20 % behind (few groups of many tokens), the mean 0.6 %.
// Warps and tiles in us, and the megabytes, the assignments a group: 16 x 2 of 16, 3328 -> 1024 -> 1024 28 and 34 (126, 2.3);
// 14 x 2 of 7, 4096 -> 1024 -> 4096 29 and 39 (116, 4); 52 x 2 of 26, 1024 -> 2048 -> 1024 50 and 46 (215, 4); 64 x 4 of 16,
// 3328 -> 2048 -> 1024 96 and 59 (285, 16); 1 x 2 of 16, 3328 -> 1024 -> 1024 14 and 25 (18, 1); 48 x 4 of 64, 1024 -> 2048 -> 1024 88 and
// 80 (513, 3); 182 x 2 of 25, fp32, 832 -> 304 -> 2312 39 and 27 (48, 15); 512 of 1, 4096 wide 249 and 131 (67, 512).
bool many_weights(int64_t tokens, int32_t k, int32_t experts, int32_t x_dtype, int64_t in_width, int64_t hidden, int64_t out_width, int32_t activation)
{
    const double groups = experts * (1.0 - std::pow(1.0 - (double)std::min(k, experts) / experts, (double)tokens));
    const double up = groups * hidden * in_width * (activation == EMB_ACT_SWIGLU ? 2 : 1) * 2e-6, down = groups * hidden * out_width * 2e-6;
    const double saved = (up + down) * (0.01 + 0.0075 * (double)(tokens * k) / groups) + (x_dtype == EMB_F32 ? 0.05 * up : 0.0);
    return saved > 0.002 * (double)(in_width + hidden);
}

// Warps that share a tile's k: as many as keep eight warps of every SM busy, but four
// steps of k for each.  (8 x 2 of 16, 3328 -> 1024 -> 1024: 26 us; for four warps 34, for sixteen 30.)
int sharing(int64_t tiles, int64_t k)
{
    int share = 1;
    while (share < kWarps && tiles * share < kSms * 8 && (k / kStep) / (share * 2) >= 4) share *= 2;
    return share;
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" int emb_expert_layer_workspace(int64_t tokens, int32_t k, int64_t in_width, int64_t hidden, int64_t out_width, size_t* bytes)
{
    if (!bytes || !sizes_valid(tokens, k, in_width, hidden, out_width)) return EMB_ERR_INVALID_ARG;
    *bytes = std::max<size_t>(Room(tokens, tokens * k, in_width, hidden, out_width).all(), 256);
    return EMB_OK;
}

extern "C" int emb_expert_layer_tiles(int64_t tokens, int32_t k, int32_t experts, int32_t x_dtype, int64_t in_width, int64_t hidden,
                                      int64_t out_width, int32_t activation, int32_t* tiles)
{
    if (!tiles || !sizes_valid(tokens, k, in_width, hidden, out_width) || experts < 1 || experts > kMaxExperts || !dtype_valid(x_dtype) ||
        activation < EMB_ACT_RELU || activation > EMB_ACT_SWIGLU)
        return EMB_ERR_INVALID_ARG;
    *tiles = tokens > 0 && many_weights(tokens, k, experts, x_dtype, in_width, hidden, out_width, activation);
    return EMB_OK;
}

extern "C" int emb_expert_layer(const void* ids, int32_t id_bytes, int64_t tokens, int32_t k, int32_t experts, const void* x, int32_t x_dtype,
                                int64_t x_stride, int64_t in_width, const void* up, const void* down, int32_t dtype, int64_t hidden,
                                int64_t out_width, int32_t activation, const float* weights, void* out, int32_t out_dtype, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    size_t need = 0;
    if (emb_expert_layer_workspace(tokens, k, in_width, hidden, out_width, &need) != EMB_OK || experts < 1 ||
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
    a.weights = weights, a.out = out, a.out_dtype = out_dtype, a.act = activation;
    const Room room(tokens, tokens * k, in_width, hidden, out_width);
    unsigned char* const at = static_cast<unsigned char*>(workspace);
    a.rows = at, a.hidden_at = at + room.rows, a.y = reinterpret_cast<float*>(at + room.rows + room.hidden);
    if (!(a.status = dense_status_word())) return EMB_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t groups = std::min<int64_t>(tokens * k, experts);     // at most
    const bool tiles = many_weights(tokens, k, experts, x_dtype, in_width, hidden, out_width, activation);
    if (!tiles && tokens * k <= kSumInDown) a.done = reinterpret_cast<int*>(at + room.rows + room.hidden + room.y);
    const auto sums = [&]() -> int {
        if (a.done) return EMB_OK;
        return launch_next(layer_sum, dim3((unsigned)((out_width / 4 + kThreads - 1) / kThreads), (unsigned)tokens), kThreads, 0, st, 1, a);
    };
    if (tiles) {
        if (int rc = launch_tiles(a, x_dtype, dtype, st)) return rc;
        return sums();
    }
    const auto go = [&](auto t) -> int {
        using T = decltype(t);
        const auto launch = [&](auto kernel, int64_t width, int units, int64_t sum) {
            const int64_t tiles = groups * ((width + units - 1) / units);
            a.share = sharing(tiles, sum);
            const unsigned blocks = (unsigned)std::min<int64_t>((tiles * a.share + kWarps - 1) / kWarps, kSms * kPerSm);
            return launch_next(kernel, blocks, kThreads, 0, st, 1, a);
        };
        const auto first = [&](auto xt) -> int {
            using X = decltype(xt);
            return activation == EMB_ACT_SWIGLU ? launch(layer_up<T, X, true>, hidden, kTile / 2, in_width) : launch(layer_up<T, X, false>, hidden, kTile, in_width);
        };
        if (int rc = x_dtype == EMB_F32 ? first(float()) : first(T())) return rc;
        if (int rc = launch(layer_down<T>, out_width, kTile, hidden)) return rc;
        return sums();
    };
    return dtype == EMB_F16 ? go(__half()) : go(__nv_bfloat16());
}

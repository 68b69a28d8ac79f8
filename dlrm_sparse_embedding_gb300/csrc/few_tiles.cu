// The expert layer for a few tokens where its weights are many: tiles of 128 rows of a
// weight on the tensor cores, D[weight row][token] = A B^T.
//
// Bound by reading the weights.  A is a weight's tile, copied by TMA in steps of 64 k to a ring
// of stages that keeps some 100 KB for an SM on their way; B is the group's tokens, a multiple of 16
// of them at a time, beside it.  (With the weights as B and the tokens as rows, every step
// would copy 128 rows of tokens, most of them not the group's.)  Both kernels' B stands by
// group in memory, the tokens' rows brought there first (gather_rows) and hidden written so:
// rows that follow the group's are read with it and their columns left alone.
// A kernel's first weights are copied before the kernel before it is done.
//
// 48 tokens, 4 of 64 experts, 1024 -> 2048 -> 1024, fp16: 78 us (about 460 MB of chosen experts, 5.9 TB/s); 64, 4 of 16, 3328 ->
// 2048 -> 1024, bf16: 58 (286 MB, 4.9 TB/s); 64, 8 of 8, 2048 wide: 46 (134 MB), fewer tiles than places for CTAs.  The four kernels
// take 11 us with 64 wide weights, and a tile's way through k 3 ns an element of it (1 of 1, 3328 -> 3328 -> 64: 33 us).  A
// group of more than TOKENS reads its weights again for each TOKENS, from L2 where they fit: 256 tokens, 2 of 4, 2048 wide 48 us
// (67 MB), 512 of 1, 4096 wide 131 (67 MB).  Measured and not kept: one CTA an SM with six stages, its B brought by four
// warps (83, 81 and 70 us); the last expert's CTA adding a tile's tokens up (85, 85 and 87).
#include "few_tokens.cuh"
#include "product_core.cuh"

namespace emb {
namespace few {
namespace {

using core::kMaxDevices;

constexpr int kRows = 128;          // of a weight's tile
constexpr int kStep = 64;           // k of a stage
constexpr int kBytesA = kRows * 128;
constexpr int kExchange = 64 * 33;  // floats: a gated tile's upper half, 32 columns at a time
constexpr int kThreads = 256;       // warps: copies, products, tensor memory, (none), epilogue
constexpr int kEpilogue = 128;      // threads

// TOKENS of a group at once.  Two CTAs of an SM share its memory, so that one's end or beginning is
// the other's middle; 128 tokens take it all.
template <int TOKENS_>
struct Shape {
    static constexpr int TOKENS = TOKENS_, kPerSm = TOKENS == 64 ? 2 : 1, kStages = TOKENS == 64 ? 4 : 6;
    static constexpr int kBytesB = TOKENS * 128;
    static constexpr int kSizes = TOKENS == 64 ? 3 : 4;      // of B: 16, 32, 64, 128 tokens
    static constexpr uint32_t kColumns = 2 * TOKENS;
};
constexpr int kMostStages = 6, kMostSizes = 4;

struct Problem {
    Args a;
    CUtensorMap weights, rows[kMostSizes];
    bool bf16;
    int tiles;
};

struct Shared {
    uint64_t full[kMostStages], empty[kMostStages], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int gave_up;
    Groups groups;
};
template <class S>
constexpr int smem_of = 1024 + S::kStages * (kBytesA + S::kBytesB) + kExchange * (int)sizeof(float) + (int)sizeof(Shared);
static_assert(smem_of<Shape<128>> <= 227 * 1024 && 2 * (smem_of<Shape<64>> + 1024) <= 228 * 1024 && 4 * kBytesA >= kCountBytes, "the SM's shared memory");

// What every role goes through in the same order: the CTA's tiles, each with its group's
// members S::TOKENS at a time.
struct Part {
    int expert, tile, first, have;     // members first .. first + have of the sorted assignments
    __device__ int size() const { return have <= 16 ? 0 : have <= 32 ? 1 : have <= 64 ? 2 : 3; }     // of B: 16 << size
};
template <class S, class F>
__device__ __forceinline__ void each_part(const Groups& g, int tiles, F f)
{
    const int total = g.active * tiles;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const int which = item / tiles, end = g.first[which + 1];
        for (int m = g.first[which]; m < end; m += S::TOKENS) {
            const Part p{g.expert[which], item - which * tiles, m, min(end - m, S::TOKENS)};
            if (!f(p)) return;
        }
    }
}

__device__ __forceinline__ void epilogue_meets() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same, and whether all of them say so: a wait that gave up in one warp ends them all.
__device__ __forceinline__ bool epilogue_agrees(bool ok)
{
    uint32_t all;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, 1, 128, p;\nselp.u32 %0, 1, 0, q;\n}" : "=r"(all) : "r"((uint32_t)ok) : "memory");
    return all != 0;
}

// The tokens' rows in the products' type, by group: a block has an assignment, whose place is
// the number of those of smaller experts and of its own's earlier ones.  The row is on its
// way meanwhile.
constexpr int kPieces = 2;      // of 8 elements a thread has on their way

template <class T, class X>
__global__ void __launch_bounds__(kThreads) gather_rows(const Args a)
{
    wait_for_earlier();
    let_next_begin();      // after the wait: what stood before this kernel is there for the next ones' first reads
    const int p = blockIdx.x, P = a.tokens * a.k, pieces = a.in_width / 8;
    const X* const from = static_cast<const X*>(a.x) + (p / a.k) * a.x_stride;
    uint4 v[kPieces];
    const auto load = [&](int i) {
        if constexpr (std::is_same<T, X>::value) return reinterpret_cast<const uint4*>(from)[i];
        else {
            const float4 u = reinterpret_cast<const float4*>(from)[2 * i], w = reinterpret_cast<const float4*>(from)[2 * i + 1];
            return make_uint4(core::pack2<T>(u.x, u.y), core::pack2<T>(u.z, u.w), core::pack2<T>(w.x, w.y), core::pack2<T>(w.z, w.w));
        }
    };
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            if (i0 + j * kThreads < pieces) v[j] = load(i0 + j * kThreads);
    };
    fetch(threadIdx.x);
    const int mine = id_of(a, p, threadIdx.x == 0);
    int place = 0;
    for (int i0 = 0; i0 < P; i0 += kThreads) {
        const int i = i0 + threadIdx.x, other = i < P ? id_of(a, i, false) : -1;
        place += __syncthreads_count(other >= 0 && (other < mine || (other == mine && i < p)));
    }
    if (mine < 0) return;
    uint4* const to = reinterpret_cast<uint4*>(static_cast<T*>(a.rows) + (int64_t)place * a.in_width);
    for (int i = threadIdx.x; i < pieces; i += kPieces * kThreads) {
        if (i != threadIdx.x) fetch(i);
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            if (i + j * kThreads < pieces) to[i + j * kThreads] = v[j];
    }
}

// UP: hidden = act(up x), GATED: 64 rows of gates and the 64 of what they let through; else y = down hidden.
template <class T, bool UP, bool GATED, class S>
__global__ void __launch_bounds__(kThreads, S::kPerSm) layer_tiles(const __grid_constant__ Problem q)
{
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) unsigned char dynamic[];
    unsigned char* const stage_a = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic) + 1023) & ~uintptr_t(1023));
    unsigned char* const stage_b = stage_a + kStages * kBytesA;
    float* const exchange = reinterpret_cast<float*>(stage_b + kStages * S::kBytesB);
    Shared& s = *reinterpret_cast<Shared*>(exchange + kExchange);
    const Groups& g = s.groups;
    const Args& a = q.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kUnits = GATED ? kRows / 2 : kRows;       // outputs of a tile
    const int k = UP ? a.in_width : a.hidden, steps = (k + kStep - 1) / kStep;

    if (threadIdx.x == 0) {
        tc::prefetch_map(&q.weights);
        for (int i = 0; i < kStages; ++i) {
            tc::bar_init(tc::smem_addr(&s.full[i]), 1);
            tc::bar_init(tc::smem_addr(&s.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_addr(&s.acc_full[i]), 1);
            tc::bar_init(tc::smem_addr(&s.acc_empty[i]), kEpilogue / 32);
        }
        s.gave_up = 0;
        tc::bar_init_fence();
    }
    if (warp == 2) tc::tmem_alloc<1>(tc::smem_addr(&s.tmem), S::kColumns);
    let_next_begin();
    make_groups(a, s.groups, stage_a, false);      // the ids, and the first weights, were there before gather_rows let this kernel begin
    tc::fence_async_shared();      // the counts were in a stage
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s.tmem;
    volatile int* const gave_up = &s.gave_up;
    const auto stage_of = [&](uint32_t n, uint32_t& phase) { phase = (n / kStages) & 1; return n % kStages; };

    if (warp == 0 && tc::elect_one()) {     // copies
        uint32_t n = 0;
        bool ok = true, waited = false;
        // B's copies come after the earlier kernel's end: until then A's run up to a ring ahead
        const auto copy_b = [&](const Part& p, uint32_t step, int i) {
            const uint32_t st = step % kStages;
            tc::load_box<1>(tc::smem_addr(stage_b + st * S::kBytesB), &q.rows[p.size()], tc::smem_addr(&s.full[st]), i * kStep, p.first, 0);
        };
        each_part<S>(g, q.tiles, [&](const Part& p) {
            int late = 0;       // steps of this part whose B is not copied yet
            const auto catch_up = [&](int i) {
                wait_for_earlier();
                waited = true;
                for (; late; --late) copy_b(p, n - late, i - late);
            };
            for (int i = 0; ok && i < steps; ++i, ++n) {
                uint32_t phase;
                const uint32_t st = stage_of(n, phase);
                if (!waited && n == kStages) catch_up(i);
                if (!(ok = tc::bar_wait(tc::smem_addr(&s.empty[st]), phase ^ 1, gave_up))) break;
                const uint32_t bar = tc::smem_addr(&s.full[st]), to = tc::smem_addr(stage_a + st * kBytesA);
                tc::bar_expect(bar, kBytesA + (16 << p.size()) * 128);
                tc::load_box<1>(to, &q.weights, bar, i * kStep, p.tile * kUnits, p.expert);
                if (GATED) tc::load_box<1>(to + kBytesA / 2, &q.weights, bar, i * kStep, a.hidden + p.tile * kUnits, p.expert);
                if (waited) copy_b(p, n, i);
                else ++late;
            }
            if (!waited) catch_up(steps);       // a short part
            return ok;
        });
        // the products of every stage are done before the block ends
        for (uint32_t i = n < kStages ? 0 : n - kStages; ok && i < n; ++i) {
            uint32_t phase;
            const uint32_t st = stage_of(i, phase);
            ok = tc::bar_wait(tc::smem_addr(&s.empty[st]), phase, gave_up);
        }
        if (!ok) {      // what was copied last lands before the block ends
            const uint64_t t0 = tc::now_ns();
            while (tc::now_ns() - t0 < 2000000) {}
        }
    } else if (warp == 1 && tc::elect_one()) {      // products
        uint32_t n = 0, made = 0;
        each_part<S>(g, q.tiles, [&](const Part& p) {
            const uint32_t acc = made & 1, instr = tc::instruction(q.bf16, false, false, kRows, 16 << p.size());
            if (!tc::bar_wait(tc::smem_addr(&s.acc_empty[acc]), ((made >> 1) & 1) ^ 1, gave_up)) return false;
            tc::fence_after();
            for (int i = 0; i < steps; ++i, ++n) {
                uint32_t phase;
                const uint32_t st = stage_of(n, phase);
                if (!tc::bar_wait(tc::smem_addr(&s.full[st]), phase, gave_up)) return false;
                tc::fence_after();
                const uint64_t x = tc::operand(tc::smem_addr(stage_a + st * kBytesA), false, 0), y = tc::operand(tc::smem_addr(stage_b + st * S::kBytesB), false, 0);
                const int parts = (min(kStep, k - i * kStep) + 15) / 16;
                for (int j = 0; j < parts; ++j)
                    tc::mma<1>(tmem + acc * S::TOKENS, x + j * tc::operand_step(false), y + j * tc::operand_step(false), instr, i > 0 || j > 0);
                tc::commit<1>(tc::smem_addr(&s.empty[st]));
            }
            tc::commit<1>(tc::smem_addr(&s.acc_full[acc]));
            ++made;
            return true;
        });
    } else if (warp >= 4 && warp < 8) {     // a lane has a weight's row: all its columns
        uint32_t made = 0;
        const int w = warp & 3, row = w * 32 + lane;
        each_part<S>(g, q.tiles, [&](const Part& p) {
            const uint32_t acc = made & 1;
            if (!epilogue_agrees(tc::bar_wait_warp(tc::smem_addr(&s.acc_full[acc]), (made >> 1) & 1, gave_up))) return false;
            tc::fence_after();
            for (int c = 0; c < p.have; c += 32) {
                uint32_t v[32];
                tc::tmem_load32(tmem + acc * S::TOKENS + ((uint32_t)(w * 32) << 16) + c, v);
                if (c + 32 >= p.have) {
                    tc::fence_before();
                    if (lane == 0) tc::bar_arrive(tc::smem_addr(&s.acc_empty[acc]));
                }
                const int have = min(32, p.have - c);
                if constexpr (UP && !GATED) {
                    // eight columns side by side, and which activation it is once for all (512 of 8, 1024 -> 4096 -> 1024, gelu:
                    // 50 us, each column by itself 63)
                    const auto each = [&](auto f) {
#pragma unroll
                        for (int i0 = 0; i0 < 32; i0 += 8)
                            if (i0 < have)
#pragma unroll
                                for (int i = i0; i < i0 + 8; ++i) v[i] = __float_as_uint(f(__uint_as_float(v[i])));
                    };
                    if (a.act == EMB_ACT_RELU) each([](float z) { return activate(EMB_ACT_RELU, z); });
                    else if (a.act == EMB_ACT_GELU) each([](float z) { return activate(EMB_ACT_GELU, z); });
                    else each([](float z) { return activate(EMB_ACT_SILU, z); });
                }
                if constexpr (GATED) {
                    if (w >= 2)
#pragma unroll
                        for (int i = 0; i < 32; ++i) exchange[(row - 64) * 33 + i] = __uint_as_float(v[i]);
                    epilogue_meets();
                    const int unit = p.tile * kUnits + row;
                    if (w < 2 && unit < a.hidden)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < have)
                                static_cast<T*>(a.hidden_at)[(int64_t)(p.first + c + i) * a.hidden + unit] =
                                    from_float<T>(activate(EMB_ACT_SILU, __uint_as_float(v[i])) * exchange[row * 33 + i]);
                    epilogue_meets();
                } else if constexpr (UP) {
                    const int unit = p.tile * kUnits + row;
                    if (unit < a.hidden)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < have)
                                static_cast<T*>(a.hidden_at)[(int64_t)(p.first + c + i) * a.hidden + unit] = from_float<T>(__uint_as_float(v[i]));
                } else {
                    const int col = p.tile * kUnits + row;
                    if (col < a.out_width)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < have) a.y[(int64_t)g.member[p.first + c + i] * a.out_width + col] = __uint_as_float(v[i]);
                }
            }
            ++made;
            return true;
        });
    }
    __syncwarp();
    __syncthreads();
    wait_for_earlier();      // a block without a tile, too: what follows takes this kernel's end for both
    if (threadIdx.x == 0 && s.gave_up) atomicOr(a.status, ERRBIT_TIMEOUT);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 2) tc::tmem_free<1>(tmem, S::kColumns);
}

template <class T, bool UP, bool GATED, class S>
int launch_kernel(Problem& q, const core::Device& dev, cudaStream_t st)
{
    const Args& a = q.a;
    const int64_t k = UP ? a.in_width : a.hidden, rows = UP ? (int64_t)a.hidden * (GATED ? 2 : 1) : a.out_width, units = GATED ? kRows / 2 : kRows;
    const int dtype = q.bf16 ? EMB_BF16 : EMB_F16, assignments = a.tokens * a.k;
    if (!core::make_map(&q.weights, dtype, UP ? a.up : a.down, false, k, rows, a.experts, k, rows * k, GATED ? kRows / 2 : kRows)) return EMB_ERR_CUDA;
    for (int i = 0; i < S::kSizes; ++i)
        if (!core::make_map(&q.rows[i], dtype, UP ? a.rows : a.hidden_at, false, k, assignments, 1, k, 0, 16 << i)) return EMB_ERR_CUDA;
    q.tiles = (int)(((UP ? a.hidden : a.out_width) + units - 1) / units);
    const auto kernel = layer_tiles<T, UP, GATED, S>;
    static std::atomic<bool> sized[kMaxDevices];
    if (!sized[dev.number].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of<S>) != cudaSuccess) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        sized[dev.number].store(true, std::memory_order_relaxed);
    }
    const int64_t items = (int64_t)std::min(assignments, a.experts) * q.tiles;
    return launch_next(kernel, (unsigned)std::min<int64_t>(items, dev.sms * S::kPerSm), kThreads, smem_of<S>, st, 1, q);
}

}  // namespace

int launch_tiles(const Args& a, int x_dtype, int dtype, cudaStream_t st)
{
    const core::Device dev = core::device();
    if (!dev.sms) return EMB_ERR_CUDA;
    Problem q;
    q.a = a;
    q.bf16 = dtype == EMB_BF16;
    const auto go = [&](auto t, auto shape) -> int {
        using T = decltype(t);
        using S = decltype(shape);
        const int blocks = a.tokens * a.k;
        if (int rc = x_dtype == EMB_F32 ? launch_next(gather_rows<T, float>, blocks, kThreads, 0, st, 1, a) : launch_next(gather_rows<T, T>, blocks, kThreads, 0, st, 1, a)) return rc;
        if (int rc = a.act == EMB_ACT_SWIGLU ? launch_kernel<T, true, true, S>(q, dev, st) : launch_kernel<T, true, false, S>(q, dev, st)) return rc;
        return launch_kernel<T, false, false, S>(q, dev, st);
    };
    const auto with_shape = [&](auto t) { return a.tokens <= 64 ? go(t, Shape<64>()) : go(t, Shape<128>()); };
    return dtype == EMB_F16 ? with_shape(__half()) : with_shape(__nv_bfloat16());
}

}  // namespace few
}  // namespace emb

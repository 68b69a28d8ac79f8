// The expert layer for a few tokens where its weights are many: tiles of 128 rows of a
// weight on the tensor cores, D[weight row][token] = A B^T.
//
// Bound by reading the weights.  A is a weight's tile, copied by TMA in steps of 64 k to a ring
// of stages that keeps some 130 KB of an SM's memory traffic on its way; B is the group's tokens, a
// multiple of 16 of up to 128 at a time, beside it.  (With the weights as B and the tokens
// as rows, every step would copy 128 rows of tokens, most of them not the group's.)
//   up:   four warps bring the tokens' rows, whatever their type and places, into B's layout
//   down: hidden stands by group, so TMA copies B as well: rows that follow the group's are
//         read with it and their columns left alone
// The second kernel's first weights are copied before the first kernel is done.
#include "few_tokens.cuh"
#include "product_core.cuh"

namespace emb {
namespace few {
namespace {

using core::kMaxDevices;

constexpr int kRows = 128;          // of a weight's tile
constexpr int kStep = 64;           // k of a stage
constexpr int kMostTokens = 128;    // of a group at once
constexpr int kStages = 6;
constexpr int kBytesA = kRows * 128, kBytesB = kMostTokens * 128;
constexpr int kSizes = 4;           // of B: 16, 32, 64 and 128 tokens
constexpr int kExchange = 64 * 33;  // floats: a gated tile's upper half, 32 columns at a time
constexpr int kEpilogue = 128;      // threads
constexpr uint32_t kColumns = 2 * kMostTokens;

struct Problem {
    Args a;
    CUtensorMap weights, hidden[kSizes];
    bool bf16;
    int tiles;
};

struct Shared {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int gave_up;
    Groups groups;
};
constexpr int kSmem = 1024 + kStages * (kBytesA + kBytesB) + kExchange * (int)sizeof(float) + (int)sizeof(Shared);
static_assert(kSmem <= 227 * 1024 && kStages * (kBytesA + kBytesB) >= kCountBytes, "the SM's shared memory");

// What every role goes through in the same order: the CTA's tiles, each with its group's
// members kMostTokens at a time.
struct Part {
    int expert, tile, first, have;     // members first .. first + have of the sorted assignments
    __device__ int eights() const { return have <= 16 ? 16 : have <= 32 ? 32 : have <= 64 ? 64 : 128; }
};
template <class F>
__device__ __forceinline__ void each_part(const Groups& g, int tiles, F f)
{
    const int total = g.active * tiles;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const int which = item / tiles, end = g.first[which + 1];
        for (int m = g.first[which]; m < end; m += kMostTokens) {
            const Part p{g.expert[which], item - which * tiles, m, min(end - m, kMostTokens)};
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

template <class T, class X>
__device__ __forceinline__ uint4 convert(const X* p)
{
    if constexpr (std::is_same<T, X>::value) return *reinterpret_cast<const uint4*>(p);
    else {
        const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
        return make_uint4(core::pack2<T>(u.x, u.y), core::pack2<T>(u.z, u.w), core::pack2<T>(v.x, v.y), core::pack2<T>(v.z, v.w));
    }
}

// UP: hidden = act(up x), GATED: 64 rows of gates and the 64 of what they let through; else y = down hidden.
template <class T, class X, bool UP, bool GATED>
__global__ void __launch_bounds__(UP ? 384 : 256, 1) layer_tiles(const __grid_constant__ Problem q)
{
    extern __shared__ __align__(1024) unsigned char dynamic[];
    unsigned char* const stage_a = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic) + 1023) & ~uintptr_t(1023));
    unsigned char* const stage_b = stage_a + kStages * kBytesA;
    float* const exchange = reinterpret_cast<float*>(stage_b + kStages * kBytesB);
    Shared& s = *reinterpret_cast<Shared*>(exchange + kExchange);
    const Groups& g = s.groups;
    const Args& a = q.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kUnits = GATED ? kRows / 2 : kRows;       // outputs of a tile
    const int k = UP ? a.in_width : a.hidden, steps = (k + kStep - 1) / kStep;

    if (threadIdx.x == 0) {
        tc::prefetch_map(&q.weights);
        for (int i = 0; i < kStages; ++i) {
            tc::bar_init(tc::smem_addr(&s.full[i]), UP ? 5 : 1);     // the copies, and the four warps that bring rows
            tc::bar_init(tc::smem_addr(&s.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_addr(&s.acc_full[i]), 1);
            tc::bar_init(tc::smem_addr(&s.acc_empty[i]), kEpilogue / 32);
        }
        s.gave_up = 0;
        tc::bar_init_fence();
    }
    if (warp == 2) tc::tmem_alloc<1>(tc::smem_addr(&s.tmem), kColumns);
    if (UP) wait_for_earlier();
    let_next_begin();      // of the first kernel after its wait: what stood before it is there for the second one's first reads
    make_groups(a, s.groups, stage_a, UP && blockIdx.x == 0);
    tc::fence_async_shared();      // the counts were in a stage
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s.tmem;
    volatile int* const gave_up = &s.gave_up;
    const auto stage_of = [&](uint32_t n, uint32_t& phase) { phase = (n / kStages) & 1; return n % kStages; };

    if (warp == 0 && tc::elect_one()) {     // copies
        uint32_t n = 0;
        bool ok = true, waited = UP;
        // B's copies come after the earlier kernel's end: until then A's run up to a ring ahead
        const auto rows_of = [&](const Part& p, uint32_t step, int i) {
            const int size = p.eights();
            const CUtensorMap* const map = &q.hidden[size == 16 ? 0 : size == 32 ? 1 : size == 64 ? 2 : 3];
            const uint32_t st = step % kStages;
            tc::load_box<1>(tc::smem_addr(stage_b + st * kBytesB), map, tc::smem_addr(&s.full[st]), i * kStep, p.first, 0);
        };
        each_part(g, q.tiles, [&](const Part& p) {
            int late = 0;       // steps of this part whose B is not copied yet
            for (int i = 0; ok && i < steps; ++i, ++n) {
                uint32_t phase;
                const uint32_t st = stage_of(n, phase);
                if (!waited && n == kStages) {       // the ring is full of A: now B
                    wait_for_earlier();
                    waited = true;
                    for (; late; --late) rows_of(p, n - late, i - late);
                }
                if (!(ok = tc::bar_wait(tc::smem_addr(&s.empty[st]), phase ^ 1, gave_up))) break;
                const uint32_t bar = tc::smem_addr(&s.full[st]), to = tc::smem_addr(stage_a + st * kBytesA);
                tc::bar_expect(bar, kBytesA + (UP ? 0 : p.eights() * 128));
                if constexpr (GATED) {
                    tc::load_box<1>(to, &q.weights, bar, i * kStep, p.tile * kUnits, p.expert);
                    tc::load_box<1>(to + kBytesA / 2, &q.weights, bar, i * kStep, a.hidden + p.tile * kUnits, p.expert);
                } else {
                    tc::load_box<1>(to, &q.weights, bar, i * kStep, p.tile * kUnits, p.expert);
                }
                if constexpr (!UP) {
                    if (waited) rows_of(p, n, i);
                    else ++late;
                }
            }
            if (!UP && !waited) {       // a short part
                wait_for_earlier();
                waited = true;
                for (int i = steps - late; late; --late, ++i) rows_of(p, n - late, i);
            }
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
        each_part(g, q.tiles, [&](const Part& p) {
            const uint32_t acc = made & 1, instr = tc::instruction(q.bf16, false, false, kRows, p.eights());
            if (!tc::bar_wait(tc::smem_addr(&s.acc_empty[acc]), ((made >> 1) & 1) ^ 1, gave_up)) return false;
            tc::fence_after();
            for (int i = 0; i < steps; ++i, ++n) {
                uint32_t phase;
                const uint32_t st = stage_of(n, phase);
                if (!tc::bar_wait(tc::smem_addr(&s.full[st]), phase, gave_up)) return false;
                tc::fence_after();
                const uint64_t x = tc::operand(tc::smem_addr(stage_a + st * kBytesA), false, 0), y = tc::operand(tc::smem_addr(stage_b + st * kBytesB), false, 0);
                const int parts = (min(kStep, k - i * kStep) + 15) / 16;
                for (int j = 0; j < parts; ++j)
                    tc::mma<1>(tmem + acc * kMostTokens, x + j * tc::operand_step(false), y + j * tc::operand_step(false), instr, i > 0 || j > 0);
                tc::commit<1>(tc::smem_addr(&s.empty[st]));
            }
            tc::commit<1>(tc::smem_addr(&s.acc_full[acc]));
            ++made;
            return true;
        });
    } else if (warp >= 4 && warp < 8) {     // a lane has a weight's row: all its columns
        uint32_t made = 0;
        const int w = warp & 3, row = w * 32 + lane;
        each_part(g, q.tiles, [&](const Part& p) {
            const uint32_t acc = made & 1;
            if (!epilogue_agrees(tc::bar_wait_warp(tc::smem_addr(&s.acc_full[acc]), (made >> 1) & 1, gave_up))) return false;
            tc::fence_after();
            for (int c = 0; c < p.have; c += 32) {
                uint32_t v[32];
                tc::tmem_load32(tmem + acc * kMostTokens + ((uint32_t)(w * 32) << 16) + c, v);
                if (c + 32 >= p.have) {
                    tc::fence_before();
                    if (lane == 0) tc::bar_arrive(tc::smem_addr(&s.acc_empty[acc]));
                }
                const int have = min(32, p.have - c);
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
                                    from_float<T>(activate(a.act, __uint_as_float(v[i])) * exchange[row * 33 + i]);
                    epilogue_meets();
                } else if constexpr (UP) {
                    const int unit = p.tile * kUnits + row;
                    if (unit < a.hidden)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < have)
                                static_cast<T*>(a.hidden_at)[(int64_t)(p.first + c + i) * a.hidden + unit] = from_float<T>(activate(a.act, __uint_as_float(v[i])));
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
    } else if (UP && warp >= 8) {       // the tokens' rows to B: 8 of a row's 16-byte pieces a step, each where the 128-byte swizzle has it
        const int thread = threadIdx.x - 256, piece = thread & 7, row0 = thread >> 3;
        constexpr int kBatch = 4;       // pieces a thread has on their way, and as many it stores
        uint32_t n = 0;
        each_part(g, q.tiles, [&](const Part& p) {
            const int each = p.eights() / 16, total = steps * each;      // a thread's pieces: of rows row0, row0 + 16, ...; step by step
            uint4 ahead[2][kBatch];
            const auto fetch = [&](uint4 (&to)[kBatch], int u) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int step = (u + i) / each, r = row0 + (u + i) % each * 16, at = step * kStep + piece * 8;
                    to[i] = make_uint4(0, 0, 0, 0);
                    if (u + i < total && r < p.have && at < k)
                        to[i] = convert<T, X>(static_cast<const X*>(a.x) + (g.member[p.first + r] / a.k) * a.x_stride + at);
                }
            };
            const auto put = [&](const uint4 (&from)[kBatch], int u) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (u + i >= total) break;
                    const int step = (u + i) / each, j = (u + i) % each, r = row0 + j * 16;
                    uint32_t phase;
                    const uint32_t st = stage_of(n + step, phase);
                    if (j == 0 && !tc::bar_wait_warp(tc::smem_addr(&s.empty[st]), phase ^ 1, gave_up)) return false;
                    *reinterpret_cast<uint4*>(stage_b + st * kBytesB + r * 128 + ((piece ^ (r & 7)) * 16)) = from[i];
                    if (j + 1 == each) {
                        tc::fence_async_shared();
                        __syncwarp();
                        if (lane == 0) tc::bar_arrive(tc::smem_addr(&s.full[st]));
                    }
                }
                return true;
            };
            fetch(ahead[0], 0);
            for (int u = 0; u < total; u += 2 * kBatch) {
                fetch(ahead[1], u + kBatch);
                if (!put(ahead[0], u)) return false;
                fetch(ahead[0], u + 2 * kBatch);
                if (!put(ahead[1], u + kBatch)) return false;
            }
            n += steps;
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
    if (warp == 2) tc::tmem_free<1>(tmem, kColumns);
}

template <class T, class X, bool UP, bool GATED>
int launch_kernel(Problem& q, const core::Device& dev, cudaStream_t st)
{
    const Args& a = q.a;
    const int64_t k = UP ? a.in_width : a.hidden, rows = UP ? (int64_t)a.hidden * (GATED ? 2 : 1) : a.out_width, units = GATED ? kRows / 2 : kRows;
    const int dtype = q.bf16 ? EMB_BF16 : EMB_F16, assignments = a.tokens * a.k;
    if (!core::make_map(&q.weights, dtype, UP ? a.up : a.down, false, k, rows, a.experts, k, rows * k, GATED ? kRows / 2 : kRows)) return EMB_ERR_CUDA;
    if (!UP)
        for (int i = 0; i < kSizes; ++i)
            if (!core::make_map(&q.hidden[i], dtype, a.hidden_at, false, k, assignments, 1, k, 0, 16 << i)) return EMB_ERR_CUDA;
    q.tiles = (int)(((UP ? a.hidden : a.out_width) + units - 1) / units);
    const auto kernel = layer_tiles<T, X, UP, GATED>;
    static std::atomic<bool> sized[kMaxDevices];
    if (!sized[dev.number].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        sized[dev.number].store(true, std::memory_order_relaxed);
    }
    const int64_t items = (int64_t)std::min(assignments, a.experts) * q.tiles;
    return launch_next(kernel, (unsigned)std::min<int64_t>(items, dev.sms), UP ? 384 : 256, kSmem, st, 1, q);
}

}  // namespace

int launch_tiles(const Args& a, int x_dtype, int dtype, cudaStream_t st)
{
    const core::Device dev = core::device();
    if (!dev.sms) return EMB_ERR_CUDA;
    Problem q;
    q.a = a;
    q.bf16 = dtype == EMB_BF16;
    const bool gated = a.act == EMB_ACT_SWIGLU;
    const auto go = [&](auto t) -> int {
        using T = decltype(t);
        const auto first = [&](auto xt) {
            using X = decltype(xt);
            return gated ? launch_kernel<T, X, true, true>(q, dev, st) : launch_kernel<T, X, true, false>(q, dev, st);
        };
        if (int rc = x_dtype == EMB_F32 ? first(float()) : first(T())) return rc;
        return launch_kernel<T, T, false, false>(q, dev, st);
    };
    return dtype == EMB_F16 ? go(__half()) : go(__nv_bfloat16());
}

}  // namespace few
}  // namespace emb

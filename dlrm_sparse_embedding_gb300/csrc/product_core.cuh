// What the tensor-core kernels share: the shapes of a tile, the ring of stages,
// how operands are copied and multiplied, the host's tensor maps.
//
// A kernel is a persistent grid: each CTA, or pair of CTAs on one 256 x 256
// tile, walks a list of tiles.  One warp's thread copies 64-wide steps of A and
// B to a ring of stages, one issues the products into one of two accumulators
// in tensor memory, and eight warps take the other accumulator through the
// epilogue meanwhile.
#pragma once

#include <atomic>

#include "emb_internal.cuh"
#include "products.cuh"
#include "tensor_core.cuh"

namespace emb {
namespace core {

constexpr int kRows = 128;                      // of an operand a CTA holds a step
constexpr int kStep = 64;                       // k of a stage: 128 bytes
constexpr int kEpilogueWarps = 8;               // two to each quarter of the accumulator's lanes, half its columns each
constexpr int kThreads = 128 + 32 * kEpilogueWarps;   // warps: copy, products, tails, (none), epilogue
constexpr int kBlockBytes = 64 * 128;           // an mn-major block: 64 k of 64 m
constexpr int kOperand = kRows * 128;           // bytes of one operand a stage
constexpr int kMaxStages = 6;
constexpr int kChunk = 32;                      // columns an epilogue warp takes at once
constexpr int kMaxDevices = 64;

// Pairs move half the bytes of single CTAs for the same products; these fill the
// GPU with less work; and where even that is not enough, tiles are half as wide and
// SPLIT CTAs share a long k.
template <int CTAS_, int SPLIT_ = 1, int COLS_ = kRows * CTAS_>
struct Shape {
    static constexpr int CTAS = CTAS_, SPLIT = SPLIT_;
    static constexpr int kCluster = CTAS * SPLIT;
    static constexpr int kTile = kRows * CTAS, kCols = COLS_;   // of D
    static constexpr int kColsHeld = kCols / CTAS;   // rows of B a CTA holds a step
    static constexpr int kStages = kMaxStages;
    static constexpr int kOperandB = kColsHeld * 128;
    static constexpr int kStageBytes = kOperand + kOperandB;
    static constexpr uint32_t kColumns = 2 * kCols;   // two accumulators
    static constexpr uint32_t kBytes = CTAS * kStageBytes;   // a stage's, over the pair
    static_assert(CTAS == 1 || SPLIT == 1, "pairs do not share a tile's k");
    static_assert(kColsHeld % 64 == 0, "whole mn-major blocks");
};

struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t part[kMaxStages], peer_part[kMaxStages];   // a step whose rows past the group are still to be zeroed; the other CTA's is done
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem;
    int gave_up;
};
constexpr int kRingBytes = 512;
static_assert(sizeof(Ring) <= kRingBytes, "the ring's room");

// Shared memory: the stages on a 1024-byte boundary, the ring, then the kernel's own.
template <class S>
constexpr int smem_bytes(int own) { return 1024 + S::kStages * S::kStageBytes + kRingBytes + own; }

struct Block {
    unsigned char* stage_a;
    unsigned char* stage_b;
    Ring* ring;
    unsigned char* own;
    uint32_t rank, tmem;
    volatile int* gave_up;
};

template <class S>
__device__ __forceinline__ Block block_of(unsigned char* dynamic)
{
    Block b;
    b.stage_a = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic) + 1023) & ~uintptr_t(1023));
    b.stage_b = b.stage_a + S::kStages * kOperand;
    b.ring = reinterpret_cast<Ring*>(b.stage_b + S::kStages * S::kOperandB);
    b.own = reinterpret_cast<unsigned char*>(b.ring) + kRingBytes;
    b.gave_up = &b.ring->gave_up;
    return b;
}

// Barriers and tensor memory; the whole block, and its pair, meet here.
template <class S>
__device__ __forceinline__ void open(Block& b)
{
    const int warp = threadIdx.x >> 5;
    b.rank = S::kCluster > 1 ? tc::cluster_rank() : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            tc::bar_init(tc::smem_addr(&b.ring->full[i]), 1);
            tc::bar_init(tc::smem_addr(&b.ring->empty[i]), 1);
            tc::bar_init(tc::smem_addr(&b.ring->part[i]), 1);
            tc::bar_init(tc::smem_addr(&b.ring->peer_part[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_addr(&b.ring->acc_full[i]), 1);
            tc::bar_init(tc::smem_addr(&b.ring->acc_empty[i]), kEpilogueWarps * S::CTAS);
        }
        b.ring->gave_up = 0;
        tc::bar_init_fence();
    }
    if (warp == 2) tc::tmem_alloc<S::CTAS>(tc::smem_addr(&b.ring->tmem), S::kColumns);
    tc::fence_before();
    __syncthreads();
    if constexpr (S::kCluster > 1) tc::cluster_sync();
    tc::fence_after();
    b.tmem = b.ring->tmem;
}

template <class S>
__device__ __forceinline__ void close(const Block& b, int* status)
{
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *b.gave_up && status) atomicOr(status, ERRBIT_TIMEOUT);
    tc::fence_before();
    if constexpr (S::kCluster > 1) tc::cluster_sync();
    tc::fence_after();
    if ((threadIdx.x >> 5) == 2) tc::tmem_free<S::CTAS>(b.tmem, S::kColumns);
}

// Where the n-th step of a role stands in the ring.
template <int STAGES>
struct Slot {
    uint32_t stage, phase;
    __device__ explicit Slot(uint32_t n) : stage(n % STAGES), phase((n / STAGES) & 1) {}
};

// Copy this CTA's part of one step: its rows (columns, if mn-major) of each operand
// from m and n on.  `part`: the step is not whole yet when it has
// arrived, and goes through ring->part.
template <class S>
__device__ __forceinline__ bool copy_step(const Block& b, uint32_t step, bool part, const CUtensorMap* map_a, bool a_mn, int m, int za,
                                          const CUtensorMap* map_b, bool b_mn, int n, int zb, int k)
{
    const Slot<S::kStages> s(step);
    if (!tc::bar_wait(tc::smem_addr(&b.ring->empty[s.stage]), s.phase ^ 1, b.gave_up)) return false;
    const uint32_t to_a = tc::smem_addr(b.stage_a + s.stage * kOperand), to_b = tc::smem_addr(b.stage_b + s.stage * S::kOperandB);
    uint32_t bar;
    if (part) {
        bar = tc::smem_addr(&b.ring->part[s.stage]);
        tc::bar_expect(bar, S::kBytes / S::CTAS);
    } else {
        // the pair's first CTA expects both CTAs' bytes; the second one's may come first
        bar = tc::smem_addr(&b.ring->full[s.stage]);
        if (S::CTAS == 1 || b.rank == 0) tc::bar_expect(bar, S::kBytes);
        if (S::CTAS == 2) bar = tc::in_cta(bar, 0);
    }
    if (a_mn) {
        tc::load_box<S::CTAS>(to_a, map_a, bar, m, k, za);
        tc::load_box<S::CTAS>(to_a + kBlockBytes, map_a, bar, m + 64, k, za);
    } else {
        tc::load_box<S::CTAS>(to_a, map_a, bar, k, m, za);
    }
    if (b_mn) {
        tc::load_box<S::CTAS>(to_b, map_b, bar, n, k, zb);
        if (S::kColsHeld > 64) tc::load_box<S::CTAS>(to_b + kBlockBytes, map_b, bar, n + 64, k, zb);
    } else {
        tc::load_box<S::CTAS>(to_b, map_b, bar, k, n, zb);
    }
    return true;
}

// After the last of `steps` copies: the products of every stage are done, here
// and in the pair's other CTA, before either ends.  If a wait gave up, what was
// copied last lands before the block ends.
template <class S>
__device__ __forceinline__ void finish_copies(const Block& b, uint32_t steps, bool ok)
{
    for (uint32_t i = steps < S::kStages ? 0 : steps - S::kStages; ok && i < steps; ++i) {
        const Slot<S::kStages> s(i);
        ok = tc::bar_wait(tc::smem_addr(&b.ring->empty[s.stage]), s.phase, b.gave_up);
    }
    if (!ok) {
        const uint64_t t0 = tc::now_ns();
        while (tc::now_ns() - t0 < 2000000) {}
    }
}

// Multiply k (> 0) into accumulator number `tile` (the count of tiles so far); step
// is the count of steps before.  Of the last step, only the 16s that k reaches.
template <class S>
__device__ __forceinline__ bool multiply(const Block& b, uint32_t tile, uint32_t step, int64_t k, uint32_t instr, bool a_mn, bool b_mn)
{
    const int steps = (int)((k + kStep - 1) / kStep), last = (int)(k - (int64_t)(steps - 1) * kStep + 15) / 16;
    const uint32_t acc = tile & 1;
    if (!tc::bar_wait(tc::smem_addr(&b.ring->acc_empty[acc]), ((tile >> 1) & 1) ^ 1, b.gave_up)) return false;
    tc::fence_after();
    const uint32_t da = tc::operand_step(a_mn), db = tc::operand_step(b_mn);
    for (int i = 0; i < steps; ++i, ++step) {
        const Slot<S::kStages> s(step);
        if (!tc::bar_wait(tc::smem_addr(&b.ring->full[s.stage]), s.phase, b.gave_up)) return false;
        tc::fence_after();
        const uint64_t x = tc::operand(tc::smem_addr(b.stage_a + s.stage * kOperand), a_mn, kBlockBytes);
        const uint64_t y = tc::operand(tc::smem_addr(b.stage_b + s.stage * S::kOperandB), b_mn, kBlockBytes);
        if (i + 1 < steps) {
#pragma unroll
            for (int j = 0; j < kStep / 16; ++j) tc::mma<S::CTAS>(b.tmem + acc * S::kCols, x + j * da, y + j * db, instr, i > 0 || j > 0);
        } else {
            for (int j = 0; j < last; ++j) tc::mma<S::CTAS>(b.tmem + acc * S::kCols, x + j * da, y + j * db, instr, i > 0 || j > 0);
        }
        tc::commit<S::CTAS>(tc::smem_addr(&b.ring->empty[s.stage]));
    }
    tc::commit<S::CTAS>(tc::smem_addr(&b.ring->acc_full[acc]));
    return true;
}

// An epilogue warp's part of accumulator number `tile`.
struct Part {
    uint32_t tmem;                 // its lanes, from the accumulator's first column on
    uint32_t full, phase, empty;   // barriers: there, and taken (the pair's first CTA's)
    int row, c0, c1;               // its 32 rows of the CTA's 128; its columns
};

template <class S>
__device__ __forceinline__ Part part_of(const Block& b, uint32_t tile)
{
    const int warp = threadIdx.x >> 5, w = warp & 3;
    const uint32_t acc = tile & 1;
    Part p;
    p.tmem = b.tmem + acc * S::kCols + ((uint32_t)(w * 32) << 16);
    p.full = tc::smem_addr(&b.ring->acc_full[acc]);
    p.phase = (tile >> 1) & 1;
    p.empty = tc::smem_addr(&b.ring->acc_empty[acc]);
    if (S::CTAS == 2) p.empty = tc::in_cta(p.empty, 0);
    p.row = w * 32;
    p.c0 = (warp - 4) / 4 * (S::kCols / 2);
    p.c1 = p.c0 + S::kCols / 2;
    return p;
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y)
{
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline Encode encoder()
{
    static std::atomic<void*> found{nullptr};
    void* f = found.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<Encode>(f);
}

// A stack of matrices in memory, copied in boxes of 64 columns: the operand's
// `held` rows at a time where its k runs along memory, 64 k at a time where not.
// What lies outside a matrix is read as zeros.
inline bool make_map(CUtensorMap* map, int dtype, const void* p, bool mn_major, int64_t cols, int64_t nrows, int64_t stack, int64_t ld,
                     int64_t stack_stride, int held = kRows)
{
    const Encode encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)nrows, (cuuint64_t)stack};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(stack > 1 ? stack_stride : ld) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(mn_major ? kStep : held), 1}, ones[3] = {1, 1, 1};
    return encode(map, dtype == EMB_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device's number (-1: none) and its SMs.
struct Device {
    int number = -1, sms = 0;
};
inline Device device()
{
    static std::atomic<int> known[kMaxDevices];
    Device d;
    if (cudaGetDevice(&d.number) != cudaSuccess || d.number < 0 || d.number >= kMaxDevices) return Device();
    d.sms = known[d.number].load(std::memory_order_relaxed);
    if (!d.sms) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, d.number) != cudaSuccess) return Device();
        known[d.number].store(d.sms, std::memory_order_relaxed);
    }
    return d;
}

}  // namespace core
}  // namespace emb

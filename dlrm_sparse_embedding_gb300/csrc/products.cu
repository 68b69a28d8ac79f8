// Matrix products of the expert layer and of the orthogonalisation, on the
// tensor cores.
//
// A persistent grid: each CTA, or pair of CTAs on one 256 x 256 tile, walks the
// tiles of all problems.  One warp's thread copies 64-wide steps of A and B to a
// ring of stages, one issues the products into one of two accumulators in
// tensor memory, and four warps take the other accumulator through the epilogue
// meanwhile.
//
// Groups of rows start anywhere and have any length.  Where they are m, a tile
// reads whatever follows its group and does not store it: a row's garbage stays
// in its row.  Where they are k (a weight's gradient), the last step's rows past
// the group are zeroed in shared memory, in both operands, before it is
// multiplied: 0 times an infinity or a NaN of the next group would not be 0.
#include <atomic>

#include "emb_internal.cuh"
#include "products.cuh"
#include "tensor_core.cuh"

namespace emb {
namespace {

constexpr int kRows = 128;                      // of A a CTA holds a step: its accumulator's lanes
constexpr int kStep = 64;                       // k of a stage: 128 bytes
constexpr int kEpilogueWarps = 8;               // two to each quarter of the accumulator's lanes, half its columns each
constexpr int kThreads = 128 + 32 * kEpilogueWarps;   // warps: copy, products, tails, (none), epilogue
constexpr int kBlockBytes = 64 * 128;           // an mn-major block: 64 k of 64 m
constexpr int kStageOperand = kRows * 128;      // bytes of one operand a stage
constexpr int kStages = 6;
constexpr int kChunk = 32;                      // columns an epilogue warp takes at once
constexpr int kStagingGroup = 32 * kChunk * 2;  // bytes of shared memory a warp takes them through, 16-bit
constexpr int kStagingStep = 32 * kChunk * 4;   // or fp32
constexpr int kMaxDevices = 64;

template <int CTAS_, int BN_>
struct Shape {
    static constexpr int CTAS = CTAS_;
    static constexpr int BM = kRows * CTAS, BN = BN_;
    static constexpr int kBRows = BN / CTAS;    // of B a CTA holds a step
    static constexpr uint32_t kColumns = 2 * BN;   // two accumulators
};

struct Control {
    uint64_t full[kStages], empty[kStages];
    uint64_t part[kStages], peer_part[kStages];   // a step whose rows past the group are still to be zeroed; the other CTA's is done
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem;
    int gave_up;
};

// What follows the sum.
enum Finish {
    kGroup,     // rounded to 16 bits: the experts' products
    kGram,      // A = s X X^T
    kQuadratic, // B = alpha A A + beta A + diagonal I
    kUpdate,    // X' = s (B X + beta X)
};

// Grouped problems need their tables, the others' sums pass as fp32.
constexpr int tail_bytes(bool group)
{
    return group ? kEpilogueWarps * kStagingGroup + 2 * (kMaxExperts + 2) * 4 : kEpilogueWarps * kStagingStep;
}
constexpr int smem_bytes(bool group) { return 1024 + kStages * 2 * kStageOperand + 512 + tail_bytes(group); }
static_assert(smem_bytes(true) <= 227 * 1024 && smem_bytes(false) <= 227 * 1024, "the SM's shared memory");

struct Tile {
    int problem;         // B's (and D's) index in its stack
    int64_t m0, m_end;   // rows of D
    int64_t n0;
    int64_t k0, k_end;
    int steps;
};

struct Problems {
    ProductArgs p;
    CUtensorMap a, b;
    int tiles_n, tiles_m;   // of one problem; tiles_m of k-grouped and batched ones
    int* status;
};

// The list of tiles.  m-grouped problems have as many tiles as their rows need,
// one problem after another, and last the rows without an expert.
template <class S>
struct List {
    const Problems& q;
    const int* start;    // m-grouped: first row tile of each group, the tail's and the end; shared memory
    const int* rows;     // grouped: first row of each group, the tail's and the end
    int64_t total;

    __device__ Tile at(int64_t t) const
    {
        Tile r;
        const int64_t row_tile = t / q.tiles_n;
        r.n0 = (t - row_tile * q.tiles_n) * S::BN;
        r.k0 = 0, r.k_end = q.p.k;
        if (q.p.m_grouped) {
            int lo = 0, hi = (int)q.p.batch;   // the last group that starts at or before row_tile
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (start[mid] <= row_tile) lo = mid; else hi = mid - 1;
            }
            r.problem = lo;
            r.m0 = rows[lo] + (row_tile - start[lo]) * S::BM;
            r.m_end = rows[lo + 1];
            if (lo == q.p.batch) r.k_end = 0;
        } else {
            r.problem = (int)(row_tile / q.tiles_m);
            r.m0 = (row_tile - (int64_t)r.problem * q.tiles_m) * S::BM;
            r.m_end = q.p.m;
            if (q.p.k_grouped) r.k0 = rows[r.problem], r.k_end = rows[r.problem + 1];
        }
        r.steps = (int)((r.k_end - r.k0 + kStep - 1) / kStep);
        return r;
    }
};

// Both tables, by the whole block: rows is the plan's offsets made sound, start
// the running count of row tiles.
template <class S>
__device__ void make_tables(const Problems& q, int* start, int* rows)
{
    const int E = (int)q.p.batch, P = (int)(q.p.m_grouped ? q.p.m : q.p.k);
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int carried = 0, tiles = 0;
        for (int base = 0; base <= E; base += 32) {   // offsets never decrease: a running maximum
            const int e = base + lane;
            int v = e <= E ? plan_offset(q.p.offsets, e, P) : P;
            v = max(v, carried);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v = max(v, u);
            }
            if (e <= E) rows[e] = v;
            carried = __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) rows[E + 1] = P;
        __syncwarp();
        for (int base = 0; base <= E; base += 32) {
            const int e = base + lane;
            const int mine = e <= E ? (rows[e + 1] - rows[e] + S::BM - 1) / S::BM : 0;
            int s = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += u;
            }
            if (e <= E) start[e] = tiles + s - mine;
            tiles += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) start[E + 1] = tiles;
    }
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

__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// The columns [c0, c1) of a tile of the experts' products.  A lane has one row's
// 32 columns; through shared memory four lanes get to store 64 bytes of a row
// each time.
template <class T>
__device__ __forceinline__ void finish_group(const ProductArgs& p, uint32_t tmem, bool empty, unsigned char* mine, int64_t m_first, int rows,
                                             int64_t n0, int c0, int c1, uint32_t acc_empty)
{
    const int lane = threadIdx.x & 31, r0 = lane >> 2, q = lane & 3;
    T* const d = static_cast<T*>(p.d) + (m_first + r0) * p.ldd + n0 + q * 8;
    for (int c = c0; c < c1; c += kChunk) {
        if (!empty) {
            uint32_t v[32];
            tc::tmem_load32(tmem + c, v);
            if (c + kChunk == c1) {
                tc::fence_before();
                if (lane == 0) tc::bar_arrive(acc_empty);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(v[8 * i + j]);
                *reinterpret_cast<uint4*>(mine + lane * 64 + ((i ^ ((lane >> 1) & 3)) * 16)) = pack8<T>(x);
            }
            __syncwarp();
        }
        const bool in = n0 + c + q * 8 < p.n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + r0;
            uint4 o = make_uint4(0, 0, 0, 0);
            if (!empty) o = *reinterpret_cast<const uint4*>(mine + r * 64 + ((q ^ ((r >> 1) & 3)) * 16));
            if (in && r < rows) *reinterpret_cast<uint4*>(d + i * 8 * p.ldd + c) = o;
        }
        __syncwarp();
    }
}

// The same for a step of the orthogonalisation: a lane's four pieces of eight
// columns, in rows r0 + 8 i, meet C there and leave again.  C for the next
// columns is on its way meanwhile.
template <Finish F>
__device__ __forceinline__ void finish_step(const ProductArgs& p, uint32_t tmem, float* mine, int64_t problem, int64_t m_first, int rows,
                                            int64_t n0, int c0, int c1, uint32_t acc_full, uint32_t phase, uint32_t acc_empty,
                                            volatile int* gave_up)
{
    const int lane = threadIdx.x & 31, r0 = lane >> 2, q = lane & 3;
    const int64_t at_c = problem * p.batch_c + (m_first + r0) * p.ldc + n0 + q * 8;
    const int64_t at_d = problem * p.batch_d + (m_first + r0) * p.ldd + n0 + q * 8;
    const __half* const c_high = static_cast<const __half*>(p.c) + at_c;
    const __half* const c_low = static_cast<const __half*>(p.c_low) + at_c;
    float s = 1.f;
    if (F != kQuadratic && p.scale) {
        s = p.scale[problem];
        if (F == kGram) s *= s;
    }
    uint4 h[4], l[4];
    const auto fetch = [&](int c) {
        const bool in = n0 + c + q * 8 < p.n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool has = in && r0 + 8 * i < rows;
            if (F != kGram) h[i] = has ? *reinterpret_cast<const uint4*>(c_high + i * 8 * p.ldc + c) : make_uint4(0, 0, 0, 0);
            if (F == kUpdate) l[i] = has ? *reinterpret_cast<const uint4*>(c_low + i * 8 * p.ldc + c) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch(c0);
    if (!tc::bar_wait(acc_full, phase, gave_up)) return;
    tc::fence_after();
    const bool wide = (p.ldd & 7) == 0 && (p.batch_d & 7) == 0 && (reinterpret_cast<uintptr_t>(p.d) & 15) == 0;
    for (int c = c0; c < c1; c += kChunk) {
        uint32_t v[32];
        tc::tmem_load32(tmem + c, v);
        if (c + kChunk == c1) {
            tc::fence_before();
            if (lane == 0) tc::bar_arrive(acc_empty);
        }
        // 16-byte piece i of row r is at i ^ (r & 7) ^ 2 (r >> 3): rows, and columns of eight rows, without conflicts
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(mine + lane * kChunk + ((i ^ (lane & 7) ^ ((lane >> 3) << 1)) * 4)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        __syncwarp();
        const bool in = n0 + c + q * 8 < p.n;
        uint4 high[4], low[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) high[i] = h[i], low[i] = l[i];
        if (c + kChunk < c1) fetch(c + kChunk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + r0, turn = (r & 7) ^ ((r >> 3) << 1);
            const float4 x = *reinterpret_cast<const float4*>(mine + r * kChunk + (((2 * q) ^ turn) * 4));
            const float4 y = *reinterpret_cast<const float4*>(mine + r * kChunk + (((2 * q + 1) ^ turn) * 4));
            float o[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            if (F == kGram) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] *= s;
            } else {
                float cv[8];
                unpack8(high[i], cv);
                if (F == kUpdate) {
                    float lv[8];
                    unpack8(low[i], lv);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = s * __fmaf_rn(p.beta, __fmaf_rn(1.f / kLowScale, lv[j], cv[j]), o[j]);
                } else {
                    const int64_t on = m_first + r - (n0 + c + q * 8);   // which of them is on the diagonal
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __fmaf_rn(p.beta, cv[j], p.alpha * o[j]) + (on == j ? p.diagonal : 0.f);
                }
            }
            if (!in || r >= rows) continue;
            if (F == kUpdate && p.d_dtype == EMB_BF16) {
                __nv_bfloat16* const d = static_cast<__nv_bfloat16*>(p.d) + at_d + i * 8 * p.ldd + c;
                if (wide) {
                    *reinterpret_cast<uint4*>(d) = pack8<__nv_bfloat16>(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n0 + c + q * 8 + j < p.n) d[j] = __float2bfloat16_rn(o[j]);
                }
                continue;
            }
            const uint4 packed = pack8<__half>(o);
            *reinterpret_cast<uint4*>(static_cast<__half*>(p.d) + at_d + i * 8 * p.ldd + c) = packed;
            if (F == kUpdate) {
                float back[8];
                unpack8(packed, back);
#pragma unroll
                for (int j = 0; j < 8; ++j) back[j] = kLowScale * (o[j] - back[j]);
                *reinterpret_cast<uint4*>(static_cast<__half*>(p.d_low) + at_d + i * 8 * p.ldd + c) = pack8<__half>(back);
            }
        }
        __syncwarp();
    }
}

template <class S, bool A_MN, bool B_MN, Finish F>
__global__ void __launch_bounds__(kThreads, 1) product_tiles(const __grid_constant__ Problems q)
{
    constexpr int CTAS = S::CTAS;
    constexpr int kBBytes = S::kBRows * 128;
    constexpr uint32_t kTx = CTAS * (kStageOperand + kBBytes);
    extern __shared__ __align__(1024) unsigned char dynamic[];
    unsigned char* const base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic) + 1023) & ~uintptr_t(1023));
    unsigned char* const stage_a = base;
    unsigned char* const stage_b = base + kStages * kStageOperand;
    Control* const ctl = reinterpret_cast<Control*>(base + 2 * kStages * kStageOperand);
    unsigned char* const staging = reinterpret_cast<unsigned char*>(ctl) + 512;
    int* const start = reinterpret_cast<int*>(staging + kEpilogueWarps * kStagingGroup);   // grouped problems only
    int* const rows = start + kMaxExperts + 2;
    static_assert(sizeof(Control) <= 512, "the control block's room");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? tc::cluster_rank() : 0;
    volatile int* const gave_up = &ctl->gave_up;

    if (warp == 0 && lane == 0) {
        tc::prefetch_map(&q.a);
        tc::prefetch_map(&q.b);
        for (int i = 0; i < kStages; ++i) {
            tc::bar_init(tc::smem_addr(&ctl->full[i]), 1);
            tc::bar_init(tc::smem_addr(&ctl->peer_part[i]), 1);
            tc::bar_init(tc::smem_addr(&ctl->empty[i]), 1);
            tc::bar_init(tc::smem_addr(&ctl->part[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_addr(&ctl->acc_full[i]), 1);
            tc::bar_init(tc::smem_addr(&ctl->acc_empty[i]), kEpilogueWarps * CTAS);
        }
        ctl->gave_up = 0;
        tc::bar_init_fence();
    }
    if (warp == 2) tc::tmem_alloc<CTAS>(tc::smem_addr(&ctl->tmem), S::kColumns);
    if (F == kGroup) make_tables<S>(q, start, rows);
    tc::fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = ctl->tmem;

    List<S> list{q, start, rows, 0};
    list.total = (q.p.m_grouped ? (int64_t)start[q.p.batch + 1] : q.p.batch * q.tiles_m) * q.tiles_n;
    const int64_t first = blockIdx.x / CTAS, step = gridDim.x / CTAS;
    const bool tails = q.p.k_grouped;

    if (warp == 0 && tc::elect_one()) {
        // copies
        uint32_t n = 0;
        bool ok = true;
        for (int64_t t = first; ok && t < list.total; t += step) {
            const Tile tile = list.at(t);
            const int za = q.p.m_grouped || q.p.k_grouped ? 0 : tile.problem, zb = q.p.k_grouped ? 0 : tile.problem;
            const int m = (int)tile.m0 + (int)rank * kRows, nn = (int)tile.n0 + (int)rank * S::kBRows;
            for (int i = 0; i < tile.steps; ++i, ++n) {
                const uint32_t s = n % kStages, phase = (n / kStages) & 1;
                if (!tc::bar_wait(tc::smem_addr(&ctl->empty[s]), phase ^ 1, gave_up)) { ok = false; break; }
                const int k = (int)tile.k0 + i * kStep;
                const uint32_t a = tc::smem_addr(stage_a + s * kStageOperand), b = tc::smem_addr(stage_b + s * kStageOperand);
                const bool part = tails && k + kStep > tile.k_end;
                uint32_t bar;
                if (part) {
                    bar = tc::smem_addr(&ctl->part[s]);
                    tc::bar_expect(bar, kTx / CTAS);
                } else {
                    // the pair's first CTA expects both CTAs' bytes; the second one's may come first
                    bar = tc::in_cta(tc::smem_addr(&ctl->full[s]), 0);
                    if (rank == 0) tc::bar_expect(tc::smem_addr(&ctl->full[s]), kTx);
                }
                if constexpr (A_MN) {
                    for (int j = 0; j < kRows / 64; ++j) tc::load_box<CTAS>(a + j * kBlockBytes, &q.a, bar, m + 64 * j, k, za);
                } else {
                    tc::load_box<CTAS>(a, &q.a, bar, k, m, za);
                }
                if constexpr (B_MN) {
                    for (int j = 0; j < S::kBRows / 64; ++j) tc::load_box<CTAS>(b + j * kBlockBytes, &q.b, bar, nn + 64 * j, k, zb);
                } else {
                    tc::load_box<CTAS>(b, &q.b, bar, k, nn, zb);
                }
            }
        }
        // the last products of every stage are done, here and in the pair's other CTA, before either ends
        for (uint32_t i = n < kStages ? 0 : n - kStages; ok && i < n; ++i)
            ok = tc::bar_wait(tc::smem_addr(&ctl->empty[i % kStages]), (i / kStages) & 1, gave_up);
        if (!ok) {   // what was copied last lands before the block ends
            const uint64_t t0 = tc::now_ns();
            while (tc::now_ns() - t0 < 2000000) {}
        }
    } else if (warp == 1 && rank == 0 && tc::elect_one()) {
        // products
        constexpr uint32_t kInstr = tc::instruction(false, A_MN, B_MN, S::BM, S::BN), kInstrBf16 = tc::instruction(true, A_MN, B_MN, S::BM, S::BN);
        const uint32_t instr = q.p.dtype == EMB_BF16 ? kInstrBf16 : kInstr;
        uint32_t n = 0, made = 0;
        bool ok = true;
        for (int64_t t = first; ok && t < list.total; t += step) {
            const Tile tile = list.at(t);
            if (!tile.steps) continue;
            const uint32_t acc = made & 1, acc_phase = (made >> 1) & 1;
            ++made;
            if (!tc::bar_wait(tc::smem_addr(&ctl->acc_empty[acc]), acc_phase ^ 1, gave_up)) break;
            tc::fence_after();
            for (int i = 0; i < tile.steps; ++i, ++n) {
                const uint32_t s = n % kStages, phase = (n / kStages) & 1;
                if (!tc::bar_wait(tc::smem_addr(&ctl->full[s]), phase, gave_up)) { ok = false; break; }
                tc::fence_after();
                const uint64_t a = tc::operand(tc::smem_addr(stage_a + s * kStageOperand), A_MN, kBlockBytes);
                const uint64_t b = tc::operand(tc::smem_addr(stage_b + s * kStageOperand), B_MN, kBlockBytes);
#pragma unroll
                for (int j = 0; j < kStep / 16; ++j)
                    tc::mma<CTAS>(tmem + acc * S::BN, a + j * tc::operand_step(A_MN), b + j * tc::operand_step(B_MN), instr, i > 0 || j > 0);
                tc::commit<CTAS>(tc::smem_addr(&ctl->empty[s]));
            }
            if (ok) tc::commit<CTAS>(tc::smem_addr(&ctl->acc_full[acc]));
        }
    } else if (warp == 2 && tails) {
        // zero the rows past a group in its last step, then hand the step on
        uint32_t n = 0, parts[kStages] = {};
        bool ok = true;
        for (int64_t t = first; ok && t < list.total; t += step) {
            const Tile tile = list.at(t);
            const int left = (int)((tile.k_end - tile.k0) % kStep);
            if (tile.steps && left) {
                const uint32_t s = (n + tile.steps - 1) % kStages;
                uint32_t turn = 0;
#pragma unroll
                for (int i = 0; i < kStages; ++i)
                    if (i == (int)s) turn = parts[i]++;
                ok = tc::bar_wait(tc::smem_addr(&ctl->part[s]), turn & 1, gave_up);   // the same in every lane
                if (ok) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    for (int j = 0; j < kRows / 64; ++j)
                        for (int i = left * 128 + lane * 16; i < kBlockBytes; i += 512)
                            *reinterpret_cast<uint4*>(stage_a + s * kStageOperand + j * kBlockBytes + i) = zero;
                    for (int j = 0; j < S::kBRows / 64; ++j)
                        for (int i = left * 128 + lane * 16; i < kBlockBytes; i += 512)
                            *reinterpret_cast<uint4*>(stage_b + s * kStageOperand + j * kBlockBytes + i) = zero;
                    tc::fence_async();
                    __syncwarp();
                    if (rank) {
                        if (lane == 0) tc::bar_arrive(tc::in_cta(tc::smem_addr(&ctl->peer_part[s]), 0));
                    } else {
                        if (CTAS == 2) ok = tc::bar_wait(tc::smem_addr(&ctl->peer_part[s]), turn & 1, gave_up);
                        if (ok && lane == 0) tc::bar_arrive(tc::smem_addr(&ctl->full[s]));
                    }
                }
            }
            n += tile.steps;
        }
    } else if (warp >= 4) {
        // epilogue: a warp has 32 rows (those of the tensor memory it can read) and half the columns
        const int w = warp & 3, c0 = (warp - 4) / 4 * (S::BN / 2), c1 = c0 + S::BN / 2;
        uint32_t made = 0;
        for (int64_t t = first; t < list.total && !*gave_up; t += step) {
            const Tile tile = list.at(t);
            const int64_t m_first = tile.m0 + (int64_t)rank * kRows + w * 32, left = tile.m_end - m_first;
            const int have = left < 0 ? 0 : left > 32 ? 32 : (int)left;
            const uint32_t acc = made & 1, acc_phase = (made >> 1) & 1;
            const uint32_t full = tc::smem_addr(&ctl->acc_full[acc]), empty = tc::in_cta(tc::smem_addr(&ctl->acc_empty[acc]), 0);
            const uint32_t mine = tmem + acc * S::BN + ((uint32_t)(w * 32) << 16);
            if (tile.steps) ++made;
            if constexpr (F == kGroup) {
                if (tile.steps) {
                    if (!tc::bar_wait(full, acc_phase, gave_up)) break;
                    tc::fence_after();
                }
                ProductArgs p = q.p;
                if (tails) p.d = static_cast<uint16_t*>(p.d) + tile.problem * p.batch_d;
                unsigned char* const room = staging + (warp - 4) * kStagingGroup;
                if (p.dtype == EMB_BF16)
                    finish_group<__nv_bfloat16>(p, mine, !tile.steps, room, m_first, have, tile.n0, c0, c1, empty);
                else
                    finish_group<__half>(p, mine, !tile.steps, room, m_first, have, tile.n0, c0, c1, empty);
            } else {
                finish_step<F>(q.p, mine, reinterpret_cast<float*>(staging + (warp - 4) * kStagingStep), tile.problem, m_first, have, tile.n0, c0, c1,
                               full, acc_phase, empty, gave_up);
            }
        }
    }

    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up && q.status) atomicOr(q.status, ERRBIT_TIMEOUT);
    tc::fence_before();
    if constexpr (CTAS == 2) tc::cluster_sync();
    tc::fence_after();
    if (warp == 2) tc::tmem_free<CTAS>(tmem, S::kColumns);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
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

// A stack of matrices in memory, copied in boxes of 64 columns; what lies
// outside a matrix is read as zeros.
bool make_map(CUtensorMap* map, int dtype, const void* p, int64_t cols, int64_t nrows, int64_t stack, int64_t ld, int64_t stack_stride, int box_rows)
{
    const Encode encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)nrows, (cuuint64_t)stack};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(stack > 1 ? stack_stride : ld) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, ones[3] = {1, 1, 1};
    return encode(map, dtype == EMB_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int multiprocessors()
{
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <class S, bool A_MN, bool B_MN, Finish F>
int launch(Problems& q, cudaStream_t st)
{
    const ProductArgs& p = q.p;
    const int sms = multiprocessors();
    q.status = dense_status_word();
    if (!sms || !q.status) return EMB_ERR_CUDA;
    const int64_t stack_a = p.m_grouped || p.k_grouped ? 1 : p.batch, stack_b = p.k_grouped ? 1 : p.batch;
    if (!(A_MN ? make_map(&q.a, p.dtype, p.a, p.m, p.k, stack_a, p.lda, p.batch_a, kStep) : make_map(&q.a, p.dtype, p.a, p.k, p.m, stack_a, p.lda, p.batch_a, kRows)) ||
        !(B_MN ? make_map(&q.b, p.dtype, p.b, p.n, p.k, stack_b, p.ldb, p.batch_b, kStep) : make_map(&q.b, p.dtype, p.b, p.k, p.n, stack_b, p.ldb, p.batch_b, S::kBRows)))
        return EMB_ERR_CUDA;
    q.tiles_n = (int)((p.n + S::BN - 1) / S::BN);
    q.tiles_m = (int)((p.m + S::BM - 1) / S::BM);
    // m-grouped: every group may add a partly filled tile, and the tail one
    const int64_t tiles = (p.m_grouped ? q.tiles_m + p.batch + 1 : q.tiles_m * p.batch) * q.tiles_n;
    const int blocks = (int)(tiles < sms / S::CTAS ? tiles : sms / S::CTAS) * S::CTAS;
    auto* const kernel = product_tiles<S, A_MN, B_MN, F>;
    static std::atomic<bool> sized[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return EMB_ERR_CUDA;
    if (!sized[dev].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(F == kGroup)) != cudaSuccess) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        sized[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(F == kGroup);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)S::CTAS, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, q) != cudaSuccess) {
        cudaGetLastError();
        return EMB_ERR_CUDA;
    }
    return EMB_OK;
}

// The combinations that the callers have.
template <class S>
int launch_shape(Problems& q, cudaStream_t st)
{
    const ProductArgs& p = q.p;
    if (p.m_grouped) return p.b_mn ? launch<S, false, true, kGroup>(q, st) : launch<S, false, false, kGroup>(q, st);
    if (p.k_grouped) return launch<S, true, true, kGroup>(q, st);
    if (!p.c) return p.a_mn ? launch<S, true, true, kGram>(q, st) : launch<S, false, false, kGram>(q, st);
    if (!p.c_low) return launch<S, false, false, kQuadratic>(q, st);
    return p.b_mn ? launch<S, false, true, kUpdate>(q, st) : launch<S, false, false, kUpdate>(q, st);
}

}  // namespace

int launch_product(const ProductArgs& p, cudaStream_t st)
{
    if (p.m_grouped && !p.b_mn && p.m <= kFewRows) return launch_few_rows(p, st);
    Problems q;
    q.p = p;
    // pairs of CTAs on 256 x 256 tiles move half the bytes of single ones on
    // 128 x 128; these fill the GPU with less work
    const int64_t big = ((p.m + 255) / 256) * ((p.n + 255) / 256) * (p.m_grouped ? 1 : p.batch);
    if (big >= 76 && !(p.m_grouped && p.m < 128 * p.batch)) return launch_shape<Shape<2, 256>>(q, st);
    return launch_shape<Shape<1, 128>>(q, st);
}

}  // namespace emb

using namespace emb;

namespace {

bool linear_valid(const emb_expert_plan* plan, int64_t in_width, int64_t out_width, int dtype)
{
    return expert_plan_valid(plan) && (dtype == EMB_F16 || dtype == EMB_BF16) && in_width >= 8 && out_width >= 8 &&
           in_width % 8 == 0 && out_width % 8 == 0 && in_width <= (1 << 24) && out_width <= (1 << 24);
}

bool array_valid(const void* p, int64_t stride, int64_t width, int64_t n)
{
    return (p || n == 0) && aligned_to(p, 16) && stride >= width && stride % 8 == 0;
}

}  // namespace

extern "C" int emb_expert_linear(const emb_expert_plan* plan, const void* rows, int64_t rows_stride, const void* weight,
                                 int64_t in_width, int64_t out_width, int32_t dtype, void* y, void* stream)
{
    if (!linear_valid(plan, in_width, out_width, dtype) || !array_valid(rows, rows_stride, in_width, plan->tokens) ||
        !array_valid(weight, in_width, in_width, 1) || !array_valid(y, out_width, out_width, plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    ProductArgs p;
    p.dtype = p.d_dtype = dtype;
    p.a = rows, p.lda = rows_stride;
    p.b = weight, p.ldb = in_width, p.batch_b = in_width * out_width;
    p.m = plan->tokens * plan->k, p.n = out_width, p.k = in_width;
    p.offsets = plan->offsets, p.m_grouped = true, p.batch = plan->experts;
    p.d = y, p.ldd = out_width;
    return launch_product(p, static_cast<cudaStream_t>(stream));
}

extern "C" int emb_expert_linear_grad_rows(const emb_expert_plan* plan, const void* grad_y, int64_t grad_stride, const void* weight,
                                           int64_t in_width, int64_t out_width, int32_t dtype, void* grad_rows, void* stream)
{
    if (!linear_valid(plan, in_width, out_width, dtype) || !array_valid(grad_y, grad_stride, out_width, plan->tokens) ||
        !array_valid(weight, in_width, in_width, 1) || !array_valid(grad_rows, in_width, in_width, plan->tokens))
        return EMB_ERR_INVALID_ARG;
    if (plan->tokens == 0) return EMB_OK;
    ProductArgs p;
    p.dtype = p.d_dtype = dtype;
    p.a = grad_y, p.lda = grad_stride;
    p.b = weight, p.ldb = in_width, p.b_mn = true, p.batch_b = in_width * out_width;
    p.m = plan->tokens * plan->k, p.n = in_width, p.k = out_width;
    p.offsets = plan->offsets, p.m_grouped = true, p.batch = plan->experts;
    p.d = grad_rows, p.ldd = in_width;
    return launch_product(p, static_cast<cudaStream_t>(stream));
}

extern "C" int emb_expert_linear_grad_weight(const emb_expert_plan* plan, const void* grad_y, int64_t grad_stride,
                                             const void* rows, int64_t rows_stride, int64_t in_width, int64_t out_width,
                                             int32_t dtype, void* grad_weight, void* stream)
{
    if (!linear_valid(plan, in_width, out_width, dtype) || !array_valid(grad_y, grad_stride, out_width, plan->tokens) ||
        !array_valid(rows, rows_stride, in_width, plan->tokens) || !array_valid(grad_weight, in_width, in_width, 1))
        return EMB_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (plan->tokens == 0)
        return cudaMemsetAsync(grad_weight, 0, (size_t)plan->experts * in_width * out_width * 2, st) == cudaSuccess ? EMB_OK : EMB_ERR_CUDA;
    ProductArgs p;
    p.dtype = p.d_dtype = dtype;
    p.a = grad_y, p.lda = grad_stride, p.a_mn = true;
    p.b = rows, p.ldb = rows_stride, p.b_mn = true;
    p.m = out_width, p.n = in_width, p.k = plan->tokens * plan->k;
    p.offsets = plan->offsets, p.k_grouped = true, p.batch = plan->experts;
    p.d = grad_weight, p.ldd = in_width, p.batch_d = in_width * out_width;
    return launch_product(p, st);
}

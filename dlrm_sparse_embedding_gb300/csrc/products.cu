// The experts' products on the tensor cores: D = A B^T for each group of rows.
//
// Bound by the tensor cores where groups are long: three products of 65536 rows,
// 1024 x 4096, 32 groups take 319, 309 and 308 us (forward, gradients of the rows and
// of the weights: 1.69, 1.74 and 1.75 PFLOP/s, the tensor cores busy 89, 93 and 86%
// of the time), and one dense product of that size by the vendor's library 280 us.  Tiles
// of 256 x 256 by pairs of CTAs are what lets them: a step of 64 k takes 512 cycles
// of products and moves 32 KB to each SM; 128 x 128 would move as much in half the
// cycles.  Where groups are short it is bound by the weights' bytes: 192 rows, 64
// experts, 1024 x 2048 take 41 us, 6.3 TB/s.
//
// Sums are fp32, cut off instead of rounded: 6e-9 of a sum of one sign for each of its
// terms (3.9e-4 at 65536).  Taking the accumulator to registers now and then, as
// short sides of the orthogonalisation do, would need a tile's 128 sums a thread there.
//
// Groups of rows start anywhere and have any length.  Where they are m, a tile
// reads whatever follows its group and does not store it: a row's garbage stays
// in its row.  Where they are k (a weight's gradient), the last step's rows past
// the group are zeroed in shared memory, in both operands, before it is
// multiplied: 0 times an infinity or a NaN of the next group would not be 0.
#include <algorithm>
#include <climits>

#include "product_core.cuh"

namespace emb {
namespace {

using namespace core;

constexpr int kStaging = 32 * kChunk * 2;       // bytes of shared memory an epilogue warp takes its columns through
constexpr int kSmem = smem_bytes<Shape<1>>(kEpilogueWarps * kStaging + 2 * (kMaxExperts + 2) * (int)sizeof(int));
static_assert(kSmem <= 227 * 1024, "the SM's shared memory");

struct Tile {
    int problem;         // the weight's index
    int64_t m0, m_end;   // rows of D
    int64_t n0;
    int cols;
    int64_t k0, k_end;
    int steps;
};

struct Problems {
    ProductArgs p;
    CUtensorMap a, b;
    int tiles_n, tiles_m;   // tiles_m of a k-grouped problem
    int* status;
};

// The list of tiles.  m-grouped problems have as many tiles as their rows need,
// one problem after another, and last the rows without an expert.  k-grouped ones
// come longest first and are dealt out back and forth, so that all CTAs get about as
// many steps (in the plan's order the tensor cores of some were busy 55% of the
// time, of others 87%).
template <class S, bool K_GROUPED>
struct List {
    const Problems& q;
    const int* start;    // first row tile of each group, the tail's and the end; k-grouped: the groups, longest first
    const int* rows;     // first row of each group, the tail's and the end; both in shared memory
    int64_t whole, total;   // tiles that are, and all of them

    // `at_once`: CTAs or pairs.  Where the last round would keep at most half of them,
    // its tiles are halves: a pair's step is bound by its products, which halve.
    __device__ List(const Problems& problems, const int* start_, const int* rows_, int64_t at_once) : q(problems), start(start_), rows(rows_)
    {
        total = (K_GROUPED ? (int64_t)q.p.experts * q.tiles_m : (int64_t)start[q.p.experts + 1]) * q.tiles_n;
        const int64_t last = total % at_once;
        whole = S::CTAS == 2 && 2 * last <= at_once ? total - last : total;
        total += total - whole;
    }

    __device__ Tile at(int64_t t) const
    {
        Tile r;
        const int64_t half = t < whole ? 0 : (t - whole) & 1;
        r.cols = t < whole ? S::kCols : S::kCols / 2;
        if (t >= whole) t = whole + (t - whole) / 2;
        const int64_t row_tile = t / q.tiles_n;
        r.n0 = (t - row_tile * q.tiles_n) * S::kTile + half * (S::kCols / 2);
        if constexpr (K_GROUPED) {
            const int64_t place = row_tile / q.tiles_m;
            r.problem = start[place];
            r.m0 = (row_tile - place * q.tiles_m) * S::kTile;
            r.m_end = q.p.m;
            r.k0 = rows[r.problem], r.k_end = rows[r.problem + 1];
        } else {
            int lo = 0, hi = q.p.experts;   // the last group that starts at or before row_tile
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (start[mid] <= row_tile) lo = mid; else hi = mid - 1;
            }
            r.problem = lo;
            r.m0 = rows[lo] + (int64_t)(row_tile - start[lo]) * S::kTile;
            r.m_end = rows[lo + 1];
            r.k0 = 0, r.k_end = lo == q.p.experts ? 0 : q.p.k;
        }
        if (r.n0 >= q.p.n) r.k_end = r.k0;   // half a tile past the columns: nothing to store
        r.steps = (int)((r.k_end - r.k0 + kStep - 1) / kStep);
        return r;
    }
};

// Which tiles of the list a CTA (a pair) takes: one a round.  Where rounds go from
// the longest groups to the shortest, every other round is dealt out backwards.
template <bool BACK_AND_FORTH>
struct Turns {
    int64_t count, mine;
    __device__ int64_t at(int64_t round) const { return round * count + (BACK_AND_FORTH && (round & 1) ? count - 1 - mine : mine); }
};

// Both tables, by the first warp: rows is the plan's offsets made sound, start the
// running count of row tiles.
template <class S>
__device__ void make_tables(const Problems& q, int* start, int* rows)
{
    const int E = q.p.experts, P = (int)(q.p.k_grouped ? q.p.k : q.p.m);
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
            const int mine = e <= E ? (int)(((int64_t)rows[e + 1] - rows[e] + S::kTile - 1) / S::kTile) : 0;
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

// An epilogue warp's columns of a tile.  A lane has one row's 32 columns;
// through shared memory four lanes get to store 64 bytes of a row each time.
// Without steps there is no accumulator: zeros are stored.
template <class T>
__device__ __forceinline__ void finish(const ProductArgs& p, const Part& part, bool empty, unsigned char* mine, int64_t at, int rows, int64_t n0)
{
    const int lane = threadIdx.x & 31, r0 = lane >> 2, q = lane & 3;
    T* const d = static_cast<T*>(p.d) + at + r0 * p.ldd + n0 + q * 8;
    for (int c = part.c0; c < part.c1; c += kChunk) {
        if (!empty) {
            uint32_t v[32];
            tc::tmem_load32(part.tmem + c, v);
            if (c + kChunk == part.c1) {
                tc::fence_before();
                if (lane == 0) tc::bar_arrive(part.empty);
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

// A's and B's majors, and whether the groups are k: forward (k, k, no), gradient
// of the rows (k, mn, no), of the weights (mn, mn, yes).
template <class S, bool A_MN, bool B_MN, bool K_GROUPED>
__global__ void __launch_bounds__(kThreads, 1) expert_products(const __grid_constant__ Problems q)
{
    extern __shared__ __align__(1024) unsigned char dynamic[];
    Block b = block_of<S>(dynamic);
    unsigned char* const staging = b.own;
    int* const start = reinterpret_cast<int*>(staging + kEpilogueWarps * kStaging);
    int* const rows = start + kMaxExperts + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_map(&q.a);
        tc::prefetch_map(&q.b);
    }
    open<S>(b);
    let_next_begin();
    wait_for_earlier();
    make_tables<S>(q, start, rows);
    __syncthreads();
    if (K_GROUPED) {
        for (int e = threadIdx.x; e < q.p.experts; e += kThreads) {   // a group's place: how many are longer
            const int mine = rows[e + 1] - rows[e];
            int place = 0;
            for (int i = 0; i < q.p.experts; ++i) {
                const int other = rows[i + 1] - rows[i];
                place += other > mine || (other == mine && i < e);
            }
            start[place] = e;
        }
        __syncthreads();
    }

    const Turns<K_GROUPED> turns{(int64_t)gridDim.x / S::CTAS, (int64_t)blockIdx.x / S::CTAS};
    const List<S, K_GROUPED> list(q, start, rows, turns.count);
    const int64_t total = list.total;

    if (warp == 0 && tc::elect_one()) {
        uint32_t n = 0;
        bool ok = true;
        for (int64_t turn = 0; ok && turns.at(turn) < total; ++turn) {
            const Tile tile = list.at(turns.at(turn));
            // (a coordinate past the rows is read as zeros, and so is the largest one)
            const int m = (int)min(tile.m0 + b.rank * kRows, (int64_t)INT_MAX), nn = (int)tile.n0 + (int)b.rank * (tile.cols / S::CTAS);
            for (int i = 0; ok && i < tile.steps; ++i, ++n) {
                const int64_t k = tile.k0 + (int64_t)i * kStep;
                ok = copy_step<S>(b, n, K_GROUPED && k + kStep > tile.k_end, &q.a, A_MN, m, 0, &q.b, B_MN, nn, K_GROUPED ? 0 : tile.problem, (int)k);
            }
        }
        finish_copies<S>(b, n, ok);
    } else if (warp == 1 && b.rank == 0 && tc::elect_one()) {
        uint32_t n = 0, made = 0;
        for (int64_t turn = 0; turns.at(turn) < total; ++turn) {
            const Tile tile = list.at(turns.at(turn));
            if (!tile.steps) continue;
            const uint32_t instr = tc::instruction(q.p.dtype == EMB_BF16, A_MN, B_MN, S::kTile, tile.cols);
            if (!multiply<S>(b, made++, n, tile.k_end - tile.k0, instr, A_MN, B_MN)) break;
            n += tile.steps;
        }
    } else if (warp == 2 && K_GROUPED) {
        // zero the rows past a group in its last step, then hand the step on
        uint32_t n = 0, times[S::kStages] = {};
        bool ok = true;
        for (int64_t turn = 0; ok && turns.at(turn) < total; ++turn) {
            const Tile tile = list.at(turns.at(turn));
            const int left = (int)((tile.k_end - tile.k0) % kStep);
            if (tile.steps && left) {
                const uint32_t s = (n + tile.steps - 1) % S::kStages;
                uint32_t time = 0;   // how many times this stage held such a step before
#pragma unroll
                for (int i = 0; i < S::kStages; ++i)
                    if (i == (int)s) time = times[i]++;
                ok = tc::bar_wait_warp(tc::smem_addr(&b.ring->part[s]), time & 1, b.gave_up);
                if (ok) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    const int end = (left + 15) / 16 * 16 * 128;   // what is multiplied
                    for (int j = 0; j < 2; ++j)
                        for (int i = j * kBlockBytes + left * 128 + lane * 16; i < j * kBlockBytes + end; i += 512) {
                            *reinterpret_cast<uint4*>(b.stage_a + s * kOperand + i) = zero;
                            *reinterpret_cast<uint4*>(b.stage_b + s * kOperand + i) = zero;
                        }
                    tc::fence_async_shared();
                    __syncwarp();
                    if (b.rank) {
                        if (lane == 0) tc::bar_arrive_cluster(tc::in_cta(tc::smem_addr(&b.ring->peer_part[s]), 0));
                    } else {
                        if (S::CTAS == 2) ok = tc::bar_wait_cluster(tc::smem_addr(&b.ring->peer_part[s]), time & 1, b.gave_up);
                        if (ok && lane == 0) tc::bar_arrive(tc::smem_addr(&b.ring->full[s]));
                    }
                }
            }
            n += tile.steps;
        }
    } else if (warp >= 4) {
        uint32_t made = 0;
        unsigned char* const mine = staging + (warp - 4) * kStaging;
        for (int64_t turn = 0; turns.at(turn) < total; ++turn) {
            const Tile tile = list.at(turns.at(turn));
            Part part = part_of<S>(b, made);
            if (tile.cols < S::kCols) part.c0 /= 2, part.c1 = part.c0 + tile.cols / 2;
            if (tile.steps) {
                ++made;
                if (!tc::bar_wait_warp(part.full, part.phase, b.gave_up)) break;
                tc::fence_after();
            }
            const int64_t m = tile.m0 + b.rank * kRows + part.row, left = tile.m_end - m;
            const int have = left < 0 ? 0 : left > 32 ? 32 : (int)left;
            const int64_t at = (K_GROUPED ? tile.problem * q.p.m : 0) * q.p.ldd + m * q.p.ldd;
            if (q.p.dtype == EMB_BF16)
                finish<__nv_bfloat16>(q.p, part, !tile.steps, mine, at, have, tile.n0);
            else
                finish<__half>(q.p, part, !tile.steps, mine, at, have, tile.n0);
        }
    }
    close<S>(b, q.status);
}

template <class S, bool A_MN, bool B_MN, bool K_GROUPED>
int launch(Problems& q, cudaStream_t st)
{
    const ProductArgs& p = q.p;
    const Device dev = device();
    q.status = dense_status_word();
    if (!dev.sms || !q.status) return EMB_ERR_CUDA;
    if (!make_map(&q.a, p.dtype, p.a, A_MN, A_MN ? p.m : p.k, A_MN ? p.k : p.m, 1, p.lda, 0) ||
        !make_map(&q.b, p.dtype, p.b, B_MN, B_MN ? p.n : p.k, B_MN ? p.k : p.n, K_GROUPED ? 1 : p.experts, p.ldb, p.n * p.k))
        return EMB_ERR_CUDA;
    q.tiles_n = (int)((p.n + S::kTile - 1) / S::kTile);
    q.tiles_m = (int)((p.m + S::kTile - 1) / S::kTile);
    // m-grouped: every group may add a partly filled tile, and the tail one
    const int64_t tiles = (K_GROUPED ? (int64_t)q.tiles_m * p.experts : q.tiles_m + p.experts + 1) * q.tiles_n;
    const int blocks = (int)std::min<int64_t>(tiles * S::CTAS, dev.sms / S::CTAS) * S::CTAS;   // pairs: two halves of a tile
    auto* const kernel = expert_products<S, A_MN, B_MN, K_GROUPED>;
    static std::atomic<bool> sized[kMaxDevices];
    if (!sized[dev.number].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        sized[dev.number].store(true, std::memory_order_relaxed);
    }
    return launch_next(kernel, blocks, kThreads, kSmem, st, S::CTAS, q);
}

template <class S>
int launch_shape(Problems& q, cudaStream_t st)
{
    if (q.p.k_grouped) return launch<S, true, true, true>(q, st);
    return q.p.b_mn ? launch<S, false, true, false>(q, st) : launch<S, false, false, false>(q, st);
}

// About how long a product takes with tiles of `tile` on `units` CTAs or pairs, in
// 64-wide steps: a step takes either the same, it is bound by its 32 KB from L2,
// and `fixed` more go by at a tile's ends.  How the rows are dealt out to the groups
// is not known here: a group is taken to end in the middle of a tile.
double estimate(const ProductArgs& p, int tile, int units, int fixed)
{
    const auto along = [&](int64_t v) { return (double)((v + tile - 1) / tile); };
    const double rows = (double)(p.k_grouped ? p.k : p.m) / p.experts, steps = (p.k_grouped ? rows : (double)p.k) / kStep;
    const double tiles_m = p.k_grouped ? along(p.m) : std::max(1.0, rows / tile + 0.5);
    return std::max(1.0, p.experts * tiles_m * along(p.n) / units) * (steps + fixed);
}

}  // namespace

int launch_product(const ProductArgs& p, cudaStream_t st)
{
    if (!p.k_grouped && !p.b_mn && p.m <= kFewRows) return launch_few_rows(p, st);
    Problems q;
    q.p = p;
    const int sms = device().sms;
    if (!sms) return EMB_ERR_CUDA;
    // Measured, single CTAs and pairs: 2488 rows, 12 groups, 1032 x 776: 17.0 and 12.0 us (1.2 rounds of tiles against 0.8);
    // 192 rows, 64 groups, 1024 x 2048: 44.2 and 47.1 us (one tile a group either way); a weight's gradient of 4096 rows,
    // 16 groups, 3328 x 1024: 45.9 and 33.5 us; 512 rows, 8 groups, 512 x 512: 5.2 and 7.2 us.
    return estimate(p, 2 * kRows, sms / 2, 10) < estimate(p, kRows, sms, 6) ? launch_shape<Shape<2>>(q, st) : launch_shape<Shape<1>>(q, st);
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
    p.dtype = dtype;
    p.a = rows, p.lda = rows_stride;
    p.b = weight, p.ldb = in_width;
    p.m = plan->tokens * plan->k, p.n = out_width, p.k = in_width;
    p.offsets = plan->offsets, p.experts = plan->experts;
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
    p.dtype = dtype;
    p.a = grad_y, p.lda = grad_stride;
    p.b = weight, p.ldb = in_width, p.b_mn = true;
    p.m = plan->tokens * plan->k, p.n = in_width, p.k = out_width;
    p.offsets = plan->offsets, p.experts = plan->experts;
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
    p.dtype = dtype;
    p.a = grad_y, p.lda = grad_stride;
    p.b = rows, p.ldb = rows_stride;
    p.m = out_width, p.n = in_width, p.k = plan->tokens * plan->k;
    p.offsets = plan->offsets, p.experts = plan->experts, p.k_grouped = true;
    p.d = grad_weight, p.ldd = in_width;
    return launch_product(p, st);
}

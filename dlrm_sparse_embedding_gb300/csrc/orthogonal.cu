// Orthogonalisation of a batch of matrices by quintic Newton-Schulz steps
// (K. Jordan et al., "Muon", 2024):
//   X0 = G / (|G|_F + eps);   A = X X^T,  X <- a X + (b A + c A A) X.
//
// Three products a step.  Their operands are fp16: 11 bits where bf16 has 8, at
// the same rate.  Rounding X to fp16 would still cost much on matrices whose
// singular values fall off: the rounding of the large ones spreads over all
// directions, and every step multiplies what lies in the small ones by up to
// a.  So X is kept as the sum of two fp16 numbers (the second one scaled up, so
// that it keeps its bits where the first is subnormal), of which only the first goes
// into the products and both into the term a X: the products' part of X' lies
// in the span of the large directions, the term a X is where the small ones
// come from.  Over 128 x 256 to 1024 x 1024 matrices with flat, 1/i, 1/i^2 and
// rank-16-plus-noise spectra the result is 0.4e-3 to 1.3e-3 off the exact one
// (2-norm), below the 1.7e-3 of the output's rounding to bf16; all in bf16, it
// is 1e-2 to 1.7e-1, all in fp16 1e-3 to 2e-2.
//
// That is after five steps.  With the default coefficients, which do not converge,
// a step passes on what the earlier ones have lost: with the output's rounding 2.5e-3
// after six, 3.4e-3 after eight, 4.8e-3 after twelve and up to 2e-2 after 32.  (A, B
// and X in two numbers each in the products too, as short sides have them, would be
// three times as many.)  With coefficients that converge it stays at 1.8e-3.
//
// In the last two steps B = b A + c A A is stored as B + d I, and d X taken
// off again in fp32: there most singular values are near 1, B is near
// (b + c) I, and what is left of it after the shift is rounded at its own,
// smaller size.  (In earlier steps the shift would let the dropped low part of
// X back into the small directions.)
//
// Matrices whose short side is at most 128 go another way (orthogonal_short.cu).
//
// G is scaled by a power of two before it is rounded, exact for bf16, and the
// rest of the norm goes into the first step's factors.  X after a step is scaled
// by one too where it is small (Lift in orthogonal.cuh).
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "orthogonal.cuh"

namespace emb {
namespace {

using namespace core;

constexpr int kNormThreads = 256;
constexpr int kMaxNormBlocks = 256;   // per matrix
constexpr int kNormBlocks = 4 * 152;  // of all: four an SM (16 of 1024 x 3328: both passes 51 us, 55 with eight and 68 with 27)
constexpr int kOneBlockThreads = 1024;
constexpr int64_t kOneBlock = 8 * 8 * kOneBlockThreads;   // elements that one block reads twice sooner than two launches pass
constexpr float kRange = 256.f;       // the scaled norm is in [kRange, 2 kRange)
constexpr int kMaxLift = 250;         // beyond it X0 is below the output's range

struct Layout {
    int64_t ld, ldm, m, x_elems, a_elems;   // pitches (multiples of 8), the short side, elements a matrix
    int norm_blocks;
    size_t x[2], x_low[2], a, b, scale, lift, done, partial, total;   // byte offsets
};

Layout layout_of(int64_t batch, int64_t rows, int64_t cols)
{
    Layout l;
    l.m = std::min(rows, cols);
    l.ld = (cols + 7) / 8 * 8;
    l.ldm = (l.m + 7) / 8 * 8;
    l.x_elems = rows * l.ld;
    l.a_elems = l.m <= kShort ? kShort * kShort : l.m * l.ldm;   // W's two parts, for short sides
    const int64_t share = std::max<int64_t>(1, kNormBlocks / std::max<int64_t>(batch, 1));   // of a matrix
    l.norm_blocks = (int)std::min<int64_t>({kMaxNormBlocks, share, (rows * cols + 8 * kNormThreads - 1) / (8 * kNormThreads)});
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~size_t(255);
        return here;
    };
    for (int i = 0; i < 2; ++i) l.x[i] = take(2 * (size_t)batch * l.x_elems);
    for (int i = 0; i < 2; ++i) l.x_low[i] = take(2 * (size_t)batch * l.x_elems);
    l.a = take(2 * (size_t)batch * l.a_elems);
    l.b = take(2 * (size_t)batch * l.a_elems);
    l.scale = take(sizeof(float) * (size_t)batch);
    l.lift = take(sizeof(int) * (size_t)batch);
    l.done = take(sizeof(unsigned) * (size_t)batch);
    l.partial = take(sizeof(double) * (size_t)batch * l.norm_blocks);
    l.total = at;
    return l;
}

// Sums: double is slow here, so only one number a warp is added up in it.
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The sum of the warps' numbers (in their lane 0), in warp 0's lanes; room for one a warp.
__device__ __forceinline__ double block_sum(double of_warp, double* room)
{
    if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = of_warp;
    __syncthreads();
    return threadIdx.x < 32 ? warp_sum(threadIdx.x < blockDim.x / 32 ? room[threadIdx.x] : 0.0) : 0.0;
}

// Calls f(row, first column, the 8 values there) for the elements of a matrix that
// are this warp's: rows are dealt out warp by warp, in pieces of 256 columns.  WIDE:
// rows are whole vectors of 16 bytes; else they are read one element at a time, and
// zeros follow a row's last one.
template <bool WIDE, class T, class F>
__device__ __forceinline__ void each_piece(const T* g, int64_t row_stride, int64_t rows, int64_t cols, F f)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    const int64_t pieces = (cols + 255) / 256, step = (int64_t)gridDim.x * warps;
    const int64_t u = (int64_t)blockIdx.x * warps + (threadIdx.x >> 5);
    int64_t row = u / pieces, piece = u - row * pieces;
    const int64_t row_step = step / pieces, piece_step = step - row_step * pieces;
    using Word = typename std::conditional<WIDE, uint4, T>::type;
    constexpr int kWords = 8 * sizeof(T) / sizeof(Word);
    constexpr int kAhead = WIDE ? 4 : 2;   // pieces on their way at once
    while (row < rows) {
        Word w[kAhead][kWords];
        int64_t at_row[kAhead], at_col[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            at_row[a] = row, at_col[a] = (piece * 32 + lane) * 8;
            if (row < rows && at_col[a] < cols) {
                const Word* const p = reinterpret_cast<const Word*>(g + row * row_stride + at_col[a]);
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    if constexpr (WIDE) w[a][i] = p[i];
                    else w[a][i] = at_col[a] + i < cols ? p[i] : from_float<T>(0.f);
                }
            } else {
                at_row[a] = rows;
            }
            row += row_step, piece += piece_step;
            if (piece >= pieces) piece -= pieces, ++row;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (at_row[a] < rows) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = to_float<T>(reinterpret_cast<const T*>(w[a])[i]);
                f(at_row[a], at_col[a], v);
            }
    }
}

// This warp's sum of squares, in every lane: fp32, eight at a time, and what rounding
// takes from the running sum is added up beside it (a thread has 44 pieces of eight
// of 16 matrices of 1024 x 3328 and 8192 of one of 65536 x 65536: by itself that sum
// could be off by as many times 2^-24); in double again where the squares could leave
// fp32's range.
template <bool WIDE, class T>
__device__ __forceinline__ double squares(const T* g, int64_t row_stride, int64_t rows, int64_t cols)
{
    float s = 0.f, rest = 0.f, top = 0.f;
    each_piece<WIDE, T>(g, row_stride, rows, cols, [&](int64_t, int64_t, const float (&v)[8]) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t = __fmaf_rn(v[i], v[i], t);
            top = fmaxf(top, fabsf(v[i]));
        }
        const bool over = t > s;   // (a NaN in either stays)
        const float more = over ? t : s, less = over ? s : t, sum = __fadd_rn(more, less);
        rest = __fadd_rn(rest, __fsub_rn(less, __fsub_rn(sum, more)));
        s = sum;
    });
    s += rest;
    if (__any_sync(0xffffffffu, top > 1e15f || (top < 1e-15f && top > 0.f))) {
        double d = 0;
        each_piece<WIDE, T>(g, row_stride, rows, cols, [&](int64_t, int64_t, const float (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fma((double)v[i], (double)v[i], d);
        });
        return warp_sum(d);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

struct Input {
    int64_t batch_stride, row_stride, rows, cols;
    float eps;
    int64_t ld;              // of X
    __half *x, *x_low;
    float* scale;
    int* lift;
    unsigned* done;
    double* partial;         // norm_blocks of each matrix
    int norm_blocks;
};

// X = G 2^e as a sum of two fp16 (for 16-bit G one: its 8 or 11 bits fit, but for
// entries below 2^-24 of the norm), and the factor that makes it 2^lift G / (|G| + eps).
// Thread 0 has the sum of squares.
template <bool WIDE, class T>
__device__ __forceinline__ void put_scaled(const Input& q, const T* g, double sum_of_squares)
{
    __shared__ float factor[2];   // their product is 2^e: for numbers below fp32's normal ones it is above its range
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum_of_squares);
        int e = 0;
        if (norm > 0 && norm < INFINITY) e = max(-120, ilogbf(kRange) - ilogb(norm));
        factor[0] = ldexpf(1.f, min(e, 100));
        factor[1] = ldexpf(1.f, max(0, e - 100));
        if (blockIdx.x == 0) {
            const double share = norm / (norm + q.eps);   // |X0|
            const int lift = share > 0 && share < 0.5 ? min(kMaxLift, -ilogb(share) - 1) : 0;
            // (a zero matrix stays zero: 1 / eps, or its square in the first A, may be infinite)
            q.scale[blockIdx.y] = norm == 0 && q.eps > 0.f ? 0.f : (float)(ldexp(1.0, lift) / ldexp(norm + q.eps, e));
            q.lift[blockIdx.y] = lift;
            q.done[blockIdx.y] = 0;
        }
    }
    __syncthreads();
    const float up = factor[0], up_more = factor[1];
    const int64_t at = (int64_t)blockIdx.y * q.rows * q.ld;
    each_piece<WIDE, T>(g, q.row_stride, q.rows, q.cols, [&](int64_t row, int64_t c, const float (&v)[8]) {
        float h[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = up * v[i] * up_more;
            l[i] = kLowScale * (h[i] - __half2float(__float2half_rn(h[i])));
        }
        // rows of X start at 16 bytes and have room for whole vectors
        *reinterpret_cast<uint4*>(q.x + at + row * q.ld + c) = core::pack8<__half>(h);
        if (sizeof(T) == 4) *reinterpret_cast<uint4*>(q.x_low + at + row * q.ld + c) = core::pack8<__half>(l);
    });
}

// Sums of squares, in blocks of a fixed order, then X.
template <bool WIDE, class T>
__global__ void __launch_bounds__(kNormThreads) norm_partials(Input q, const T* __restrict__ g)
{
    __shared__ double warp_sums[kNormThreads / 32];
    let_next_begin();
    wait_for_earlier();
    const double d = block_sum(squares<WIDE, T>(g + blockIdx.y * q.batch_stride, q.row_stride, q.rows, q.cols), warp_sums);
    if (threadIdx.x == 0) q.partial[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = d;
}

template <bool WIDE, class T>
__global__ void __launch_bounds__(kNormThreads) scale_in(Input q, const T* __restrict__ g)
{
    __shared__ double warp_sums[kNormThreads / 32];
    static_assert(kMaxNormBlocks <= kNormThreads, "one partial sum a thread");
    let_next_begin();
    wait_for_earlier();
    const double d = (int)threadIdx.x < q.norm_blocks ? q.partial[(int64_t)blockIdx.y * q.norm_blocks + threadIdx.x] : 0.0;
    put_scaled<WIDE, T>(q, g + blockIdx.y * q.batch_stride, block_sum(warp_sum(d), warp_sums));
}

// Both by one block a matrix.
template <bool WIDE, class T>
__global__ void __launch_bounds__(kOneBlockThreads) norm_and_scale(Input q, const T* __restrict__ g)
{
    __shared__ double warp_sums[kOneBlockThreads / 32];
    let_next_begin();
    wait_for_earlier();
    const T* const mine = g + blockIdx.y * q.batch_stride;
    put_scaled<WIDE, T>(q, mine, block_sum(squares<WIDE, T>(mine, q.row_stride, q.rows, q.cols), warp_sums));
}

template <bool WIDE, class T>
int start(const Input& q, const T* g, int64_t batch, cudaStream_t st)
{
    if (q.rows * q.cols <= kOneBlock) return launch_next(norm_and_scale<WIDE, T>, dim3(1, (unsigned)batch), kOneBlockThreads, 0, st, 1, q, g);
    const dim3 grid(q.norm_blocks, (unsigned)batch);
    if (int rc = launch_next(norm_partials<WIDE, T>, grid, kNormThreads, 0, st, 1, q, g)) return rc;
    return launch_next(scale_in<WIDE, T>, grid, kNormThreads, 0, st, 1, q, g);
}

// ---------------------------------------------------------------------------
// the steps
// ---------------------------------------------------------------------------
// 16 matrices of 1024 x 3328 take 970 us for five steps, 950 TFLOP/s of what symmetry
// leaves: reading G twice and writing X takes 51 us of them, and of the rest the
// tensor cores are busy 52%, DRAM 63% (3.7 GB): A's products (33 thousand cycles a
// tile, 27 of them products) run beside nothing that uses memory, the update (16 and
// 8) beside 512 KB of X a tile.  One of 1777 x 519 takes 123 us,
// bound by the chain of 15 products: 7 us each, of which the products are 1 to 2.
//
// All products of all steps are one list of tiles for one persistent grid (see
// Walk).  A tile needs its own matrix's earlier tiles and no other's, so
// matrices run into each other's products instead of waiting at 3 x steps
// launches; a counter a matrix says how far it is.  CTAs take tiles in the
// list's order, and the launch is cooperative, so what a tile waits for is done
// or running.
//
// A and B are symmetric: only the tiles on and below the diagonal are computed,
// the others are written as their transposes.
//
// With few tiles they are 64 columns wide, and the k of A's (the long side) is
// shared by a cluster: every CTA sums its part of the steps, sends each other one its
// 32 rows of the sum, and finishes its own 32 rows from the parts it was sent, added
// in the CTAs' order.
enum Product { kGram, kQuadratic, kUpdate };   // A = X X^T, B = b A + c A A, X' = a X + B X

constexpr int kSplit = 4;
constexpr int kStaging = 32 * kChunk * 4;       // bytes of shared memory for 32 rows of 32 columns in fp32

struct Counts {
    int ahead;   // tiles whose C may be read
    int taken;   // tiles the epilogue has begun
    int stored[kEpilogueWarps];   // tiles each of its warps has stored
    uint64_t received, sent;      // barriers: the parts of this CTA's rows are here; the parts it sent have been used
};
constexpr int kCountsBytes = 128;
static_assert(sizeof(Counts) <= kCountsBytes, "the counts' room");

// Staging: 32 x 32 of a warp, and where tiles are shared as much again for the parts
// that come in: 32 rows of 64 columns of each CTA.
template <class S>
constexpr int staging_bytes() { return (S::SPLIT == 1 ? 1 : 2) * kEpilogueWarps * kStaging; }
using Few = Shape<1, kSplit, 64>;
static_assert(kSplit * 2 == kEpilogueWarps && kSplit * 32 == kRows, "a CTA of a cluster finishes a quarter of a tile's rows");
template <class S>
constexpr int own_smem()
{
    static_assert(smem_bytes<S>(staging_bytes<S>() + kCountsBytes) <= 227 * 1024, "the SM's shared memory");
    return smem_bytes<S>(staging_bytes<S>() + kCountsBytes);
}

struct Steps {
    // operands: x_gram of A = X X^T, x_update of X' = B X (or X B), the `n` ones in the place of B
    CUtensorMap x_gram[2], x_gram_n[2], x_update[2], a_map, a_map_n, b_map;
    __half *x[2], *x_low[2], *a, *b;
    __nv_bfloat16* out;
    const float* scale;
    Lift lift;
    unsigned* done;          // of each matrix: CTAs that have finished a tile
    int64_t rows, cols, ld, ldm, m;
    int64_t long_stride, short_stride;   // between matrices: of X, of A and B
    unsigned batch;
    int steps;
    bool tall;
    float ca, cb, cc;
    unsigned squares;        // tiles of A on and below the diagonal
    unsigned tiles_m, tiles_n;   // of X
    bool low_in;             // the first X has a low part
    int* status;
};

struct Tile {
    Product product;
    int step, matrix;
    int64_t m0, n0;
    int64_t k;
    int k_steps;             // of 64
    unsigned needs;          // of done[matrix]
};

// How many tiles a matrix has of a product, and how many CTAs finish one.
__device__ __forceinline__ unsigned tiles_of(const Steps& q, Product p)
{
    return p == kUpdate ? q.tiles_m * q.tiles_n : q.squares;
}
template <class S>
__device__ __forceinline__ constexpr unsigned finishers(Product p) { return S::CTAS * (p == kGram ? S::SPLIT : 1); }

// Tile `index` of a product, the matrices' one after another.
template <class S>
__device__ __forceinline__ Tile tile_of(const Steps& q, int step, Product product, unsigned index)
{
    Tile r;
    r.step = step;
    r.product = product;
    const unsigned gram = tiles_of(q, kGram), update = tiles_of(q, kUpdate);
    r.needs = step * (gram * (finishers<S>(kGram) + finishers<S>(kQuadratic)) + update * finishers<S>(kUpdate));
    int64_t k = q.m;
    if (product == kUpdate) {
        r.needs += gram * (finishers<S>(kGram) + finishers<S>(kQuadratic));
        r.matrix = index / update;
        const unsigned idx = index - r.matrix * update;
        r.m0 = (int64_t)(idx / q.tiles_n) * S::kTile;
        r.n0 = (int64_t)(idx % q.tiles_n) * S::kCols;
    } else {
        if (product == kGram) k = q.rows + q.cols - q.m;
        else r.needs += gram * finishers<S>(kGram);
        r.matrix = index / gram;
        const unsigned idx = index - r.matrix * gram;
        constexpr unsigned kWide = S::kTile / S::kCols;   // row i of the triangle starts at kWide i (i + 1) / 2
        unsigned i = (unsigned)((sqrtf(8.f / kWide * (float)idx + 1.f) - 1.f) * 0.5f);
        while (kWide * i * (i + 1) / 2 > idx) --i;
        while (kWide * (i + 1) * (i + 2) / 2 <= idx) ++i;
        r.m0 = (int64_t)i * S::kTile;
        r.n0 = (int64_t)(idx - kWide * i * (i + 1) / 2) * S::kCols;
    }
    r.k = k;
    r.k_steps = (int)((k + kStep - 1) / kStep);
    return r;
}

// The tiles of one CTA, in the list's order: step by step, in a step A's, B's and
// then X's, in each the matrices one after another.  Without a shared k they are
// dealt out over the whole list; with one, A's tiles go to clusters and the others
// to CTAs, product by product.  (Half the matrices half a step behind the others, so
// that products bound by memory and by the tensor cores run side by side, measured
// the same: 1044 us for 16 of 1024 x 3328, against 1016.)
template <class S>
struct Walk {
    const Steps& q;
    int step;
    int product;
    unsigned index;   // of a tile among all matrices' of the product

    __device__ explicit Walk(const Steps& steps) : q(steps), step(0), product(kGram), index(blockIdx.x / S::kCluster) { settle(); }
    __device__ bool more() const { return step < q.steps; }
    __device__ Tile tile() const { return tile_of<S>(q, step, (Product)product, index); }
    __device__ void next()
    {
        index += S::SPLIT > 1 && product != kGram ? gridDim.x : gridDim.x / S::kCluster;
        settle();
    }

private:
    __device__ void settle()
    {
        while (step < q.steps) {
            const unsigned count = q.batch * tiles_of(q, (Product)product);
            if (index < count) return;
            index -= count;
            if (++product > kUpdate) product = kGram, ++step;
            if (S::SPLIT > 1) index = product == kGram ? blockIdx.x / S::kCluster : blockIdx.x;
        }
    }
};

// Waits until a matrix has got so far; false when the limit ran out.
__device__ __forceinline__ bool wait_done(const unsigned* done, unsigned needs, volatile int* gave_up)
{
    const auto reached = [&] {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
        return (int)(v - needs) >= 0;
    };
    if (!needs || reached()) return true;
    const uint64_t start = tc::now_ns();
    while (!reached()) {
        if (*gave_up) return false;
        if (tc::now_ns() - start > tc::kWaitLimitNs) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

// Counters in shared memory, one writer each.
__device__ __forceinline__ bool wait_count(const int* count, int least, volatile int* gave_up)
{
    const auto reached = [&] {
        int v;
        asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(tc::smem_addr(count)) : "memory");
        return v >= least;
    };
    if (reached()) return true;
    const uint64_t start = tc::now_ns();
    while (!reached()) {
        if (*gave_up) return false;
        if (tc::now_ns() - start > tc::kWaitLimitNs) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void set_count(int* count, int v)
{
    asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(tc::smem_addr(count)), "r"(v) : "memory");
}

// An epilogue warp's columns of a tile.  Through shared memory (a lane has one
// row's 32 columns of the accumulator) a lane gets four pieces of eight columns,
// in rows r0 + 8 i, which meet C there and leave again.  C for the next columns
// is on its way meanwhile; it was written in this launch by other SMs, so it
// comes from L2.
//   kGram       D = s sum
//   kQuadratic  D = cc sum + cb C + diagonal I
//   kUpdate     D = s (sum + beta (C + C's low part))
// with s for X's lift, and the input's scale in the first step.
template <class S, Product F, bool SHARED = (S::SPLIT > 1 && F == kGram)>
__device__ __forceinline__ bool finish(const Steps& q, const Tile& tile, const Part& part, float* mine, uint32_t rank, unsigned parts,
                                       uint32_t received, uint32_t turn_of, volatile int* gave_up)
{
    const int c0 = part.c0, c1 = part.c1;
    const int lane = threadIdx.x & 31, r0 = lane >> 2, p = lane & 3;
    const int64_t height = F == kUpdate ? q.rows : q.m, width = F == kUpdate ? q.cols : q.m, ld = F == kUpdate ? q.ld : q.ldm;
    const int64_t m_first = tile.m0 + (S::CTAS == 2 ? rank * kRows : 0) + (SHARED ? rank * 32 : part.row), left = height - m_first;
    const int rows = left < 0 ? 0 : left > 32 ? 32 : (int)left;
    const int64_t of_matrix = tile.matrix * (F == kUpdate ? q.rows * q.ld : q.m * q.ldm);
    const int64_t at = of_matrix + (m_first + r0) * ld + tile.n0 + p * 8;
    const __half *high = nullptr, *low = nullptr;
    __half *d = nullptr, *d_low = nullptr;
    float diagonal = 0.f;   // the shift of B that the last two steps use, taken off again in their update
    if (tile.step > 0 && tile.step >= q.steps - 2) diagonal = (tile.step == q.steps - 1 ? -0.9f : -0.73f) * (q.cb + q.cc);
    const bool last = F == kUpdate && tile.step == q.steps - 1;
    if (F == kGram) {
        d = q.a + at;
    } else if (F == kQuadratic) {
        high = q.a + at;
        d = q.b + at;
    } else {
        high = q.x[tile.step & 1] + at, low = tile.step || q.low_in ? q.x_low[tile.step & 1] + at : nullptr;
        d = q.x[(tile.step + 1) & 1] + at, d_low = q.x_low[(tile.step + 1) & 1] + at;
    }
    const float beta = F == kUpdate ? q.ca - diagonal : q.cb;
    float s = 1.f;
    if (F != kQuadratic) {
        s = F == kGram ? q.lift.of_square(tile.matrix, tile.step) : q.lift.between(tile.matrix, tile.step, tile.step + 1);
        if (tile.step == 0) s *= F == kGram ? q.scale[tile.matrix] * q.scale[tile.matrix] : q.scale[tile.matrix];
    }
    const bool out_wide = (q.cols & 7) == 0 && (reinterpret_cast<uintptr_t>(q.out) & 15) == 0;
    __nv_bfloat16* const out = q.out + tile.matrix * q.rows * q.cols + (m_first + r0) * q.cols + tile.n0 + p * 8;

    uint4 h[4], l[4];
    const auto fetch = [&](int c) {
        const bool in = tile.n0 + c + p * 8 < width;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool has = in && r0 + 8 * i < rows;
            if (F != kGram) h[i] = has ? __ldcg(reinterpret_cast<const uint4*>(high + i * 8 * ld + c)) : make_uint4(0, 0, 0, 0);
            if (F == kUpdate) l[i] = has && low ? __ldcg(reinterpret_cast<const uint4*>(low + i * 8 * ld + c)) : make_uint4(0, 0, 0, 0);
        }
    };
    if (F != kGram) fetch(c0);
    if (!SHARED) {
        if (!tc::bar_wait_warp(part.full, part.phase, gave_up)) return false;
        tc::fence_after();
    } else {
        if (!tc::bar_wait_cluster(received, turn_of, gave_up)) return false;
    }
    for (int c = c0; c < c1; c += kChunk) {
        if constexpr (!SHARED) {
            uint32_t v[32];
            tc::tmem_load32(part.tmem + c, v);
            if (c + kChunk == c1) {
                tc::fence_before();
                if (lane == 0) tc::bar_arrive(part.empty);
            }
            // 16-byte piece i of row r is at i ^ (r & 7) ^ 2 (r >> 3): rows, and columns of eight rows, without conflicts
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(mine + lane * kChunk + ((i ^ (lane & 7) ^ ((lane >> 3) << 1)) * 4)) =
                    make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            __syncwarp();
        }
        const int64_t n = tile.n0 + c + p * 8;
        uint4 ch[4], cl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ch[i] = h[i], cl[i] = l[i];
        if (F != kGram && c + kChunk < c1) fetch(c + kChunk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + r0, turn = (r & 7) ^ ((r >> 3) << 1);
            float4* const px = reinterpret_cast<float4*>(mine + r * kChunk + (((2 * p) ^ turn) * 4));
            float4* const py = reinterpret_cast<float4*>(mine + r * kChunk + (((2 * p + 1) ^ turn) * 4));
            float2 o[4] = {};
            if constexpr (!SHARED) {
                const float4 x = *px, y = *py;
                o[0] = make_float2(x.x, x.y), o[1] = make_float2(x.z, x.w), o[2] = make_float2(y.x, y.y), o[3] = make_float2(y.z, y.w);
            } else {
#pragma unroll
                for (int k = 0; k < S::SPLIT; ++k)
                    if (parts >> k & 1) {   // part k, 64 columns of 32 rows further on
                        const float4 x = px[k * (2 * kStaging / 16)], y = py[k * (2 * kStaging / 16)];
                        o[0] = add2(o[0], make_float2(x.x, x.y)), o[1] = add2(o[1], make_float2(x.z, x.w));
                        o[2] = add2(o[2], make_float2(y.x, y.y)), o[3] = add2(o[3], make_float2(y.z, y.w));
                    }
            }
            if (F == kGram) {
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = mul2(both(s), o[j]);
            } else {
                float2 cv[4];
                if (F == kUpdate) {
                    join8(ch[i], cl[i], cv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = mul2(both(s), fma2(both(beta), cv[j], o[j]));
                } else {
                    unpack8(ch[i], cv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = fma2(both(beta), cv[j], mul2(both(q.cc), o[j]));
                    const int64_t on = m_first + r - n;   // which of them is on the diagonal
                    if (diagonal != 0.f && on >= 0 && on < 8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (on == 2 * j) o[j].x += diagonal;
                            if (on == 2 * j + 1) o[j].y += diagonal;
                        }
                    }
                }
            }
            if (F != kUpdate && tile.n0 + S::kCols <= tile.m0) {   // for the transpose below
                *px = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
                *py = make_float4(o[2].x, o[2].y, o[3].x, o[3].y);
            }
            if (n >= width || r >= rows) continue;
            if (last) {
                __nv_bfloat16* const to = out + i * 8 * q.cols + c;
                if (out_wide) {
                    *reinterpret_cast<uint4*>(to) = pack8<__nv_bfloat16>(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < width) to[j] = __float2bfloat16_rn(j & 1 ? o[j / 2].y : o[j / 2].x);
                }
                continue;
            }
            if (F == kUpdate) {
                uint4 top, rest;
                split8(o, top, rest);
                *reinterpret_cast<uint4*>(d + i * 8 * ld + c) = top;
                __stcs(reinterpret_cast<uint4*>(d_low + i * 8 * ld + c), rest);
            } else {
                *reinterpret_cast<uint4*>(d + i * 8 * ld + c) = pack8<__half>(o);
            }
        }
        __syncwarp();
        if (F != kUpdate && tile.n0 + S::kCols <= tile.m0) {
            // column n of these 32 rows is 32 elements of row n of the other triangle: four lanes store 64 bytes of it
            __half* const t = (F == kGram ? q.a : q.b) + of_matrix + (tile.n0 + c + r0) * ld + m_first + p * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = i * 8 + r0;
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = mine[(p * 8 + j) * kChunk + (((col >> 2) ^ j ^ (p << 1)) * 4) + (col & 3)];
                if (tile.n0 + c + col < width && p * 8 < rows) *reinterpret_cast<uint4*>(t + i * 8 * ld) = pack8<__half>(o);
            }
            __syncwarp();
        }
    }
    return true;
}

// A warp's 32 rows and columns of this CTA's part of the sum, to the CTA of those
// rows.
template <class S>
__device__ __forceinline__ bool send_part(const Block& b, Counts* counts, const Part& part, float* mine, unsigned char* received)
{
    const int lane = threadIdx.x & 31;
    const uint32_t to = part.row / 32, half = part.c0 / kChunk;
    if (!tc::bar_wait_warp(part.full, part.phase, b.gave_up)) return false;
    tc::fence_after();
    uint32_t v[32];
    tc::tmem_load32(part.tmem + part.c0, v);
    tc::fence_before();
    __syncwarp();
    if (lane == 0) tc::bar_arrive(part.empty);
    // a lane's 16 bytes at a time would cross to the other CTAs one by one (9 bytes a cycle); a 4 KB copy does not
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(mine + lane * kChunk + ((i ^ (lane & 7) ^ ((lane >> 3) << 1)) * 4)) =
            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    tc::fence_async_shared();
    __syncwarp();
    if (lane == 0)
        tc::copy_cluster(tc::in_cta(tc::smem_addr(received + (b.rank * 2 + half) * kStaging), to), tc::smem_addr(mine), kStaging,
                         tc::in_cta(tc::smem_addr(&counts->received), to));
    return true;
}

// One warp goes two tiles ahead of the epilogue: it waits until the tile's matrix is
// far enough, for the copies and the epilogue alike (each would wait 2000 cycles a
// tile for L2's answer and the fence).  (Having X brought to L2 here as well gave
// nothing for its low part and cost a tenth for its high one.)
template <class S>
__device__ __forceinline__ void scout(const Steps& q, const Block& b, Counts* s)
{
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (Walk<S> walk(q); walk.more(); walk.next(), ++n) {
        const Tile tile = walk.tile();
        if (!__all_sync(0xffffffffu, wait_count(&s->taken, n - 2, b.gave_up))) return;
        if (!__all_sync(0xffffffffu, wait_done(q.done + tile.matrix, tile.needs, b.gave_up))) return;
        if (lane == 0) {
            tc::fence_async();   // the copies to come read what other SMs' plain stores wrote
            set_count(&s->ahead, n + 1);
        }
    }
}

// This CTA's part of a tile's steps: [from, to).
template <class S>
__device__ __forceinline__ void part_steps(const Tile& tile, int rank, int& from, int& to)
{
    const bool shared = S::SPLIT > 1 && tile.product == kGram;
    from = shared ? tile.k_steps * rank / S::SPLIT : 0;
    to = shared ? tile.k_steps * (rank + 1) / S::SPLIT : tile.k_steps;
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1) newton_schulz(const __grid_constant__ Steps q)
{
    extern __shared__ __align__(1024) unsigned char dynamic[];
    Block b = block_of<S>(dynamic);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Counts* const counts = reinterpret_cast<Counts*>(b.own + staging_bytes<S>());
    if (threadIdx.x == 0) {
        counts->ahead = counts->taken = 0;
        for (int i = 0; i < kEpilogueWarps; ++i) counts->stored[i] = 0;
        tc::bar_init(tc::smem_addr(&counts->received), 1);
        tc::bar_init(tc::smem_addr(&counts->sent), 2 * S::SPLIT);
    }
    open<S>(b);

    if (warp == 0 && tc::elect_one()) {
        uint32_t n = 0;
        int begun = 0;
        bool ok = true;
        for (Walk<S> walk(q); ok && walk.more(); walk.next()) {
            const Tile tile = walk.tile();
            const int shift = S::CTAS == 2 ? (int)b.rank * kRows : 0, z = tile.matrix;
            const int m = (int)tile.m0 + shift, nn = (int)tile.n0 + shift;
            const CUtensorMap *ma = &q.a_map, *mb = &q.a_map_n;
            bool a_mn = false, b_mn = false;
            if (tile.product == kGram) {
                ma = &q.x_gram[tile.step & 1];
                mb = &q.x_gram_n[tile.step & 1];
                a_mn = b_mn = q.tall;
            } else if (tile.product == kUpdate) {
                ma = q.tall ? &q.x_update[tile.step & 1] : &q.b_map;
                mb = q.tall ? &q.b_map : &q.x_update[tile.step & 1];
                b_mn = !q.tall;
            }
            tc::prefetch_map(ma);
            tc::prefetch_map(mb);
            int from, to;
            part_steps<S>(tile, b.rank, from, to);
            ok = wait_count(&counts->ahead, ++begun, b.gave_up);
            for (int i = from; ok && i < to; ++i, ++n) ok = copy_step<S>(b, n, false, ma, a_mn, m, z, mb, b_mn, nn, z, i * kStep);
        }
        finish_copies<S>(b, n, ok);
    } else if (warp == 1 && (S::CTAS == 1 || b.rank == 0) && tc::elect_one()) {
        uint32_t n = 0, made = 0;
        for (Walk<S> walk(q); walk.more(); walk.next()) {
            const Tile tile = walk.tile();
            int from, to;
            part_steps<S>(tile, b.rank, from, to);
            if (from == to) continue;
            const bool a_mn = tile.product == kGram && q.tall, b_mn = tile.product == kGram ? q.tall : tile.product == kUpdate && !q.tall;
            const uint32_t instr = tc::instruction(false, a_mn, b_mn, S::kTile, S::kCols);
            if (!multiply<S>(b, made++, n, min(tile.k, (int64_t)to * kStep) - (int64_t)from * kStep, instr, a_mn, b_mn)) break;
            n += to - from;
        }
    } else if (warp == 2) {
        // a tile's stores, once all its warps have made them, are ordered before the matrix's count by one
        // thread: each warp waiting for its own to reach L2 would hold the epilogue up.  Eight lanes have
        // acquired a warp's count each (the vote orders no memory): they meet before that thread releases for all.
        int made = 0;
        for (Walk<S> walk(q); walk.more(); walk.next()) {
            const Tile tile = walk.tile();
            ++made;
            if (!__all_sync(0xffffffffu, wait_count(&counts->stored[lane % kEpilogueWarps], made, b.gave_up))) break;
            __syncwarp();
            if (lane == 0) {
                __threadfence();
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(q.done + tile.matrix) : "memory");
            }
        }
    } else if (warp == 3) {
        scout<S>(q, b, counts);
    } else if (warp >= 4) {
        int made = 0;
        uint32_t accumulators = 0, shared_tiles = 0;
        float* const mine = reinterpret_cast<float*>(b.own + (warp - 4) * kStaging);
        unsigned char* const in = b.own + kEpilogueWarps * kStaging;   // shared tiles: what comes from other CTAs, at any time
        const auto stored = [&] {   // this warp's stores, for the warp that tells the other SMs of them
            __syncwarp();
            if (lane == 0) set_count(&counts->stored[warp - 4], made + 1);
        };
        for (Walk<S> walk(q); walk.more(); walk.next(), ++made) {
            const Tile tile = walk.tile();
            int from, to;
            part_steps<S>(tile, b.rank, from, to);
            const Part part = part_of<S>(b, accumulators);
            if (from < to) ++accumulators;
            if (threadIdx.x == 4 * 32) set_count(&counts->taken, made + 1);
            bool ok = true;
            if (S::SPLIT > 1 && tile.product == kGram) {
                unsigned parts = 0;   // the CTAs that have one
                for (int i = 0; i < S::SPLIT; ++i) {
                    int f, t;
                    part_steps<S>(tile, i, f, t);
                    parts |= (unsigned)(f < t) << i;
                }
                const uint32_t turn = shared_tiles++ & 1;
                if (threadIdx.x == 4 * 32) tc::bar_expect(tc::smem_addr(&counts->received), __popc(parts) * 2 * kStaging);
                if (from < to) ok = send_part<S>(b, counts, part, mine, in);
                if (ok && (warp & 3) == 0) {   // a warp for each 32 of the columns
                    ok = finish<S, kGram>(q, tile, part, reinterpret_cast<float*>(in + part.c0 / kChunk * kStaging), b.rank, parts,
                                          tc::smem_addr(&counts->received), turn, b.gave_up);
                    if (ok) stored();
                    if (ok && lane < S::SPLIT) tc::bar_arrive_cluster(tc::in_cta(tc::smem_addr(&counts->sent), lane));
                } else if (ok) {
                    stored();
                }
                // every CTA has used what came from here: the room for it is free again
                ok = ok && tc::bar_wait_cluster(tc::smem_addr(&counts->sent), turn, b.gave_up);
            } else {
                ok = __all_sync(0xffffffffu, wait_count(&counts->ahead, made + 1, b.gave_up));
                if (ok)
                    ok = tile.product == kGram        ? finish<S, kGram>(q, tile, part, mine, b.rank, 1, 0, 0, b.gave_up)
                         : tile.product == kQuadratic ? finish<S, kQuadratic>(q, tile, part, mine, b.rank, 1, 0, 0, b.gave_up)
                                                      : finish<S, kUpdate>(q, tile, part, mine, b.rank, 1, 0, 0, b.gave_up);
                if (ok) stored();
            }
            if (!ok) break;
        }
    }
    close<S>(b, q.status);
}

int64_t along(int64_t v, int64_t tile) { return (v + tile - 1) / tile; }

// Tiles of rows x cols that cover a square's diagonal and what is below it.
int64_t squares(int64_t m, int64_t rows, int64_t cols)
{
    const int64_t n = along(m, rows), wide = rows / cols;
    return wide * n * (n + 1) / 2 - (wide * n - along(m, cols));
}

template <class S>
int launch_steps(Steps& q, cudaStream_t st)
{
    const Device dev = device();
    q.status = dense_status_word();
    if (!dev.sms || !q.status) return EMB_ERR_CUDA;
    q.squares = (unsigned)squares(q.m, S::kTile, S::kCols);
    q.tiles_m = (unsigned)along(q.rows, S::kTile);
    q.tiles_n = (unsigned)along(q.cols, S::kCols);
    const int64_t update = (int64_t)q.tiles_m * q.tiles_n, tiles = (2 * (int64_t)q.squares + update) * q.batch * q.steps;
    if (tiles > INT_MAX) return EMB_ERR_INVALID_ARG;
    // A's products run along the long side: X is k-major in them where its rows are long, and in the update where not
    const auto map = [&](CUtensorMap* m, const __half* x, bool mn_major, int held) {
        return make_map(m, EMB_F16, x, mn_major, q.cols, q.rows, q.batch, q.ld, q.long_stride, held);
    };
    const auto short_map = [&](CUtensorMap* m, const __half* a, int held) {
        return make_map(m, EMB_F16, a, false, q.m, q.m, q.batch, q.ldm, q.short_stride, held);
    };
    for (int i = 0; i < 2; ++i)
        if (!map(&q.x_gram[i], q.x[i], q.tall, kRows) || !map(&q.x_gram_n[i], q.x[i], q.tall, S::kColsHeld) ||
            !map(&q.x_update[i], q.x[i], !q.tall, kRows))
            return EMB_ERR_CUDA;
    // B is the first operand, or the second where the matrix is tall
    if (!short_map(&q.a_map, q.a, kRows) || !short_map(&q.a_map_n, q.a, S::kColsHeld) || !short_map(&q.b_map, q.b, q.tall ? S::kColsHeld : kRows))
        return EMB_ERR_CUDA;
    auto* const kernel = newton_schulz<S>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S::kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = own_smem<S>();
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)S::kCluster, 1, 1};
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<int> resident[kMaxDevices];   // clusters that run at the same time
    int clusters = resident[dev.number].load(std::memory_order_relaxed);
    if (!clusters) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, own_smem<S>()) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 1) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        resident[dev.number].store(clusters, std::memory_order_relaxed);
    }
    const int64_t most = q.batch * std::max<int64_t>(q.squares, update);
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(clusters, most) * S::kCluster);
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, q) != cudaSuccess) {
        cudaGetLastError();
        return EMB_ERR_CUDA;
    }
    return EMB_OK;
}

// About how long a step takes, in us.  A product starts `start` after the one before
// it (epilogue, the way over L2, the first copies) and takes `first` for each 64 of
// its k; where it has more tiles than run at once, every further round takes `more`
// for each 64 of k, or an epilogue.
template <class S>
double step_time(const Steps& q, int sms, double start, double first, double more, double epilogue)
{
    const double units = sms / S::CTAS;
    const auto product = [&](int64_t tiles, double at_once, double k) {
        k = std::ceil(k / kStep);
        return start + first * k + (std::ceil(tiles / at_once) - 1) * std::max(epilogue, more * k);
    };
    const int64_t gram = q.batch * squares(q.m, S::kTile, S::kCols), update = q.batch * along(q.rows, S::kTile) * along(q.cols, S::kCols);
    return product(gram, units / S::SPLIT, (double)(q.rows + q.cols - q.m) / S::SPLIT) + product(gram, units, (double)q.m) +
           product(update, units, (double)q.m);
}

// Measured, single CTAs, pairs and shared 64-wide tiles: one 1777 x 519 matrix 189, 232 and 126 us; one 256 x 1024 116, 138
// and 87; two 1024 x 1024 147, 204 and 164; 24 of 300 x 500 178, 215 and 289; one 3325 x 3001 667, 711 and 1119; 16 of
// 1024 x 3328 1052, 896 and 2066.  The numbers below are fitted to these and eleven more.
int run_steps(Steps& q, cudaStream_t st)
{
    const int sms = device().sms;
    if (!sms) return EMB_ERR_CUDA;
    const double single = step_time<Shape<1>>(q, sms, 5.5, 0.3, 0.19, 5), pairs = step_time<Shape<2>>(q, sms, 8.2, 0.29, 0.29, 8);
    const double few = step_time<Few>(q, sms, 5, 0.25, 0.25, 4);
    if (few < pairs && few < single) return launch_steps<Few>(q, st);
    return pairs < single ? launch_steps<Shape<2>>(q, st) : launch_steps<Shape<1>>(q, st);
}

bool sizes_valid(int64_t batch, int64_t rows, int64_t cols)
{
    return batch >= 0 && batch <= 65535 && rows >= 1 && cols >= 1 && rows <= 65536 && cols <= 65536;
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" int emb_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes)
{
    if (!bytes || !sizes_valid(batch, rows, cols)) return EMB_ERR_INVALID_ARG;
    *bytes = std::max<size_t>(256, layout_of(batch, rows, cols).total);
    return EMB_OK;
}

extern "C" int emb_orthogonalize(const void* update, int32_t dtype, int64_t batch_stride, int64_t row_stride, int64_t batch,
                                 int64_t rows, int64_t cols, int32_t steps, float a, float b, float c, float eps, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    size_t need = 0;
    if (emb_orthogonalize_workspace(batch, rows, cols, &need) != EMB_OK || !dtype_valid(dtype) || steps < 1 || steps > 32 ||
        row_stride < cols || batch_stride < 0 || !aligned_to(update, dtype_bytes(dtype)) || !aligned_to(out, 2) || !(eps >= 0.f))
        return EMB_ERR_INVALID_ARG;
    if (batch == 0) return EMB_OK;
    if (!update || !out || !workspace || !aligned_to(workspace, 256) || workspace_bytes < need) return EMB_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char* const ws = static_cast<char*>(workspace);
    const Layout l = layout_of(batch, rows, cols);
    const bool wide = cols % 8 == 0 && row_stride % 8 == 0 && batch_stride % 8 == 0 && aligned_to(update, 16);
    Input in;
    in.batch_stride = batch_stride, in.row_stride = row_stride, in.rows = rows, in.cols = cols;
    in.eps = eps, in.ld = l.ld;
    in.x = reinterpret_cast<__half*>(ws + l.x[0]);
    in.x_low = reinterpret_cast<__half*>(ws + l.x_low[0]);
    in.scale = reinterpret_cast<float*>(ws + l.scale);
    in.lift = reinterpret_cast<int*>(ws + l.lift);
    in.done = reinterpret_cast<unsigned*>(ws + l.done);
    in.partial = reinterpret_cast<double*>(ws + l.partial);
    in.norm_blocks = l.norm_blocks;
    const auto begin = [&](auto t) {
        using T = decltype(t);
        const T* const g = static_cast<const T*>(update);
        return wide ? start<true, T>(in, g, batch, st) : start<false, T>(in, g, batch, st);
    };
    const int rc = dtype == EMB_F32 ? begin(float()) : dtype == EMB_F16 ? begin(__half()) : begin(__nv_bfloat16());
    if (rc != EMB_OK) return rc;
    StepsArgs p;
    for (int i = 0; i < 2; ++i) {
        p.x[i] = reinterpret_cast<__half*>(ws + l.x[i]);
        p.x_low[i] = reinterpret_cast<__half*>(ws + l.x_low[i]);
    }
    p.low_in = dtype == EMB_F32;
    p.scale = reinterpret_cast<const float*>(ws + l.scale);
    p.lift = reinterpret_cast<const int*>(ws + l.lift);
    p.batch = batch, p.rows = rows, p.cols = cols, p.ld = l.ld;
    p.steps = steps;
    p.a = a, p.b = b, p.c = c;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.w = reinterpret_cast<__half*>(ws + l.a);
    p.w_low = reinterpret_cast<__half*>(ws + l.b);
    if (l.m <= kShort) return run_short(p, st);
    Steps q;
    q.tall = rows > cols;
    q.rows = rows, q.cols = cols, q.ld = l.ld, q.ldm = l.ldm, q.m = l.m;
    q.batch = (unsigned)batch, q.steps = steps, q.low_in = p.low_in;
    q.ca = a, q.cb = b, q.cc = c;
    for (int i = 0; i < 2; ++i) q.x[i] = p.x[i], q.x_low[i] = p.x_low[i];
    q.a = p.w, q.b = p.w_low;
    q.out = p.out;
    q.scale = p.scale;
    q.lift = lift_of(p.lift, a, steps);
    q.done = reinterpret_cast<unsigned*>(ws + l.done);
    q.short_stride = l.a_elems, q.long_stride = l.x_elems;
    return run_steps(q, st);
}

// Newton-Schulz steps on matrices whose short side m is at most 128.
//
// All steps are polynomials of A0 = X0 X0^T:
//   Q = a I + b A + c A A,   A <- Q A Q,   W <- W Q,   and at the end W X0,
// so the long side is needed at both ends only, and in between a CTA keeps its
// matrix's A, Q and W in shared memory: a step is a few products of 128 x 128,
// with no other SM to wait for.  What bounds it is the chain: 14 products of
// five steps, each of which needs the one before, 1600 cycles of tensor cores (24
// instructions of 128 x 128 x 16) and about as many of epilogue.  32 matrices of 128 x
// 256 take 45 us with the norm before and W X0 after it, 35 of them in this kernel;
// as products over memory, three a step, they took 106.
//
// W's eigenvalues grow by up to a a step where X's singular values are small,
// and their rounding must not reach the large ones.  So A, Q and W are held as
// two fp16 numbers, 22 bits, each product is three (the low parts' own product
// is below the last bit), and W may grow kGrowth-fold (five steps of a = 3.44);
// more steps are done in passes of kGrowthMany (three), with X written back in
// between, because what one pass loses the next ones multiply.  Emulated in 64 bits
// over 1 x 1 to 128 x 256 matrices of flat, 1/i, 1/i^2, low-rank and rank-1 spectra,
// the result is 1e-6 to 4e-4 off after five steps, less than the output's rounding to
// bf16 (1.7e-3), and 1e-5 after nine (in passes of five and four: up to 1e-3, six
// at once: 5e-3).  (One fp16 number for each would be far off: with so few singular
// values a rounding has few others to average with.)
#include <cmath>

#include "orthogonal.cuh"

namespace emb {
namespace {

using namespace core;

constexpr float kGrowth = 600.f, kGrowthMany = 50.f;
// The tensor cores truncate where fp32 rounds: over 5000 columns A0 was 2e-5 off,
// which W's growth made 6e-3 of the result.  After so many steps of 64 columns
// the accumulator's sum goes on in registers.
constexpr int kChain = 8;
constexpr int kMatrix = kShort * kShort * 2;   // bytes of one 128 x 128 fp16 matrix: two operands' stages of 64 k

struct Short {
    CUtensorMap x, x_low;          // of A0 = X X^T
    CUtensorMap x_apply, x_low_apply, w_map, w_low_map;
    const float* scale;            // or null for 1
    Lift lift;
    int before;                    // steps of earlier passes
    __half *w, *w_low;
    __half *x_out, *x_low_out;     // of the pass; null in the last one
    __nv_bfloat16* out;
    int64_t rows, cols, ld;
    bool tall, low_in;
    int steps, k_steps, tiles;
    float a, b, c;
    int* status;
};

// ---------------------------------------------------------------------------
// all steps of a matrix
// ---------------------------------------------------------------------------
constexpr int kWarps = 16;                       // of the epilogue: four to each quarter of the rows, 32 columns each
constexpr int kStepsThreads = 128 + 32 * kWarps;

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t done[2];    // the products into the first (second) pair of accumulators
    uint64_t drained[2]; // the epilogue's warps have added that part of A0's sum up
    uint64_t ready;      // the epilogue's warps have written what the next product reads
    uint32_t tmem;
    int gave_up;
};

// Matrices in shared memory: two blocks of 64 columns, 128 rows of 128 bytes
// with the 128-byte swizzle, as an operand is copied.
struct Matrix {
    unsigned char *high, *low;

    __device__ static uint32_t at(int row, int col) { return (col >> 6) * (kMatrix / 2) + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4); }
    __device__ void store(int row, int col, const float2 (&v)[4]) const
    {
        uint4 h, l;
        split8(v, h, l);
        *reinterpret_cast<uint4*>(high + at(row, col)) = h;
        *reinterpret_cast<uint4*>(low + at(row, col)) = l;
    }
    __device__ void load(int row, int col, float2 (&v)[4]) const
    {
        join8(*reinterpret_cast<const uint4*>(high + at(row, col)), *reinterpret_cast<const uint4*>(low + at(row, col)), v);
    }
};

// The products of one 64-wide step: x y into `tmem`, (x y_low + x_low y) into
// the accumulator after it.  Addresses in shared memory; 0: no low part.
__device__ __forceinline__ void multiply_split(uint32_t tmem, uint32_t x, uint32_t x_low, bool x_mn, uint32_t y, uint32_t y_low, bool y_mn, bool first)
{
    const uint32_t instr = tc::instruction(false, x_mn, y_mn, kRows, kRows), dx = tc::operand_step(x_mn), dy = tc::operand_step(y_mn);
    const auto run = [&](uint32_t to, uint32_t p, uint32_t r, bool fresh) {
        const uint64_t u = tc::operand(p, x_mn, kBlockBytes), v = tc::operand(r, y_mn, kBlockBytes);
#pragma unroll
        for (int j = 0; j < kStep / 16; ++j) tc::mma<1>(to, u + j * dx, v + j * dy, instr, !fresh || j > 0);
    };
    run(tmem, x, y, first);
    if (y_low) run(tmem + kRows, x, y_low, first);
    if (x_low) run(tmem + kRows, x_low, y, first && !y_low);
}

__device__ __forceinline__ void multiply_matrices(uint32_t tmem, const Matrix& x, const Matrix& y)
{
    for (int i = 0; i < 2; ++i)
        multiply_split(tmem, tc::smem_addr(x.high) + i * kOperand, tc::smem_addr(x.low) + i * kOperand, false,
                       tc::smem_addr(y.high) + i * kOperand, tc::smem_addr(y.low) + i * kOperand, false, i == 0);
}

constexpr int kStepsSmem = 1024 + 6 * kMatrix + 512;
static_assert(kMaxStages * 2 * kOperand == 6 * kMatrix, "the ring of A0's sum is the matrices' room");
static_assert(sizeof(Control) <= 512 && kStepsSmem <= 227 * 1024, "the SM's shared memory");

__global__ void __launch_bounds__(kStepsThreads, 1) short_steps(const __grid_constant__ Short q)
{
    extern __shared__ __align__(1024) unsigned char dynamic[];
    unsigned char* const base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic) + 1023) & ~uintptr_t(1023));
    Control* const ctl = reinterpret_cast<Control*>(base + 6 * kMatrix);
    const Matrix A{base, base + kMatrix}, Q{base + 2 * kMatrix, base + 3 * kMatrix}, W{base + 4 * kMatrix, base + 5 * kMatrix};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, z = blockIdx.x;
    volatile int* const gave_up = &ctl->gave_up;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            tc::bar_init(tc::smem_addr(&ctl->full[i]), 1);
            tc::bar_init(tc::smem_addr(&ctl->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_addr(&ctl->done[i]), 1);
            tc::bar_init(tc::smem_addr(&ctl->drained[i]), kWarps);
        }
        tc::bar_init(tc::smem_addr(&ctl->ready), kWarps);
        ctl->gave_up = 0;
        tc::bar_init_fence();
        tc::prefetch_map(&q.x);
    }
    if (warp == 2) tc::tmem_alloc<1>(tc::smem_addr(&ctl->tmem), 4 * kRows);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ctl->tmem;
    let_next_begin();
    wait_for_earlier();

    if (warp == 0 && tc::elect_one()) {
        // X's steps: the high part in the first half of a stage, the low part in the second
        bool ok = true;
        for (int i = 0; ok && i < q.k_steps; ++i) {
            const Slot<kMaxStages> s(i);
            ok = tc::bar_wait(tc::smem_addr(&ctl->empty[s.stage]), s.phase ^ 1, gave_up);
            if (!ok) break;
            const uint32_t to = tc::smem_addr(base + s.stage * 2 * kOperand), bar = tc::smem_addr(&ctl->full[s.stage]);
            tc::bar_expect(bar, q.low_in ? 2 * kOperand : kOperand);
            for (int part = 0; part < (q.low_in ? 2 : 1); ++part) {
                const CUtensorMap* const map = part ? &q.x_low : &q.x;
                const uint32_t at = to + part * kOperand;
                if (q.tall) {
                    tc::load_box<1>(at, map, bar, 0, i * kStep, z);
                    tc::load_box<1>(at + kBlockBytes, map, bar, 64, i * kStep, z);
                } else {
                    tc::load_box<1>(at, map, bar, i * kStep, 0, z);
                }
            }
        }
        if (!ok) {   // what was copied last lands before the block ends
            const uint64_t t0 = tc::now_ns();
            while (tc::now_ns() - t0 < 2000000) {}
        }
    } else if (warp == 1 && tc::elect_one()) {
        bool ok = true;
        uint32_t readies = 0;
        const auto wait_ready = [&] {
            ok = ok && tc::bar_wait(tc::smem_addr(&ctl->ready), readies++ & 1, gave_up);
            tc::fence_after();
            return ok;
        };
        for (int i = 0; ok && i < q.k_steps; ++i) {
            const Slot<kMaxStages> s(i);
            const int chain = i / kChain, pair = chain & 1;
            if (i % kChain == 0 && chain >= 2) ok = tc::bar_wait(tc::smem_addr(&ctl->drained[pair]), ((chain >> 1) & 1) ^ 1, gave_up);
            ok = ok && tc::bar_wait(tc::smem_addr(&ctl->full[s.stage]), s.phase, gave_up);
            if (!ok) break;
            tc::fence_after();
            const uint32_t x = tc::smem_addr(base + s.stage * 2 * kOperand), low = q.low_in ? x + kOperand : 0;
            multiply_split(tmem + pair * 2 * kRows, x, low, q.tall, x, low, q.tall, i % kChain == 0);
            tc::commit<1>(tc::smem_addr(&ctl->empty[s.stage]));
            if (i % kChain == kChain - 1 || i + 1 == q.k_steps) tc::commit<1>(tc::smem_addr(&ctl->done[pair]));
        }
        for (int i = 0; ok && i < q.steps; ++i) {
            const bool more = i + 1 < q.steps;
            if (!wait_ready()) break;
            multiply_matrices(tmem, A, A);
            tc::commit<1>(tc::smem_addr(&ctl->done[0]));
            if (!wait_ready()) break;
            if (more) {
                multiply_matrices(tmem, Q, A);
                tc::commit<1>(tc::smem_addr(&ctl->done[0]));
            }
            if (i) {
                multiply_matrices(tmem + 2 * kRows, W, Q);
                tc::commit<1>(tc::smem_addr(&ctl->done[1]));
            }
            if (more) {
                if (!wait_ready()) break;
                multiply_matrices(tmem, A, Q);   // A holds Q A
                tc::commit<1>(tc::smem_addr(&ctl->done[0]));
            }
        }
    } else if (warp >= 4) {
        // a lane has 32 columns of a row
        const int row = (warp & 3) * 32 + lane, c0 = (warp - 4) / 4 * 32;
        const bool diagonal = c0 == (warp & 3) * 32;
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t dones[2] = {};
        bool ok = true;
        const auto wait_done = [&](int pair) {
            ok = ok && tc::bar_wait_warp(tc::smem_addr(&ctl->done[pair]), dones[pair]++ & 1, gave_up);
            tc::fence_after();
            return ok;
        };
        // every eight columns of a pair of accumulators, added up
        const auto each = [&](int pair, auto f) {
            uint32_t v[32], l[32];
            tc::tmem_load32(mine + pair * 2 * kRows + c0, v);
            tc::tmem_load32(mine + pair * 2 * kRows + kRows + c0, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = fma2(both(1.f / kLowScale), make_float2(__uint_as_float(l[8 * i + 2 * j]), __uint_as_float(l[8 * i + 2 * j + 1])),
                                make_float2(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1])));
                f(c0 + 8 * i, o);
            }
        };
        const auto written = [&] {
            tc::fence_async_shared();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tc::smem_addr(&ctl->ready));
        };
        const auto to_matrix = [&](const Matrix& m) { return [&m, row](int col, const float2 (&o)[4]) { m.store(row, col, o); }; };
        const auto to_memory = [&](int col, const float2 (&o)[4]) {
            uint4 h, l;
            split8(o, h, l);
            const int64_t at = ((int64_t)z * kShort + row) * kShort + col;
            *reinterpret_cast<uint4*>(q.w + at) = h;
            *reinterpret_cast<uint4*>(q.w_low + at) = l;
        };
        {
            const float s = q.lift.of_square(z, q.before) * (q.scale ? q.scale[z] * q.scale[z] : 1.f);
            const int chains = (q.k_steps + kChain - 1) / kChain;
            float sum[32] = {};
            for (int chain = 0; chain < chains; ++chain) {
                const int pair = chain & 1;
                if (!wait_done(pair)) break;
                uint32_t v[32];
                tc::tmem_load32(mine + pair * 2 * kRows + c0, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] += __uint_as_float(v[i]);
                if (q.low_in) {
                    tc::tmem_load32(mine + pair * 2 * kRows + kRows + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[i] = __fmaf_rn(1.f / kLowScale, __uint_as_float(v[i]), sum[i]);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem_addr(&ctl->drained[pair]));
            }
            if (ok) {
#pragma unroll
                for (int c = 0; c < 32; c += 8) {
                    float2 o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = mul2(both(s), make_float2(sum[c + 2 * j], sum[c + 2 * j + 1]));
                    A.store(row, c0 + c, o);
                }
                written();
            }
        }
        for (int i = 0; ok && i < q.steps; ++i) {
            const bool more = i + 1 < q.steps;
            if (!wait_done(0)) break;
            each(0, [&](int col, float2 (&o)[4]) {
                float2 a[4];
                A.load(row, col, a);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = fma2(both(q.b), a[j], mul2(both(q.c), o[j]));
                if (diagonal) {   // a lane's own row is on it somewhere in these columns
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (col + 2 * j == row) o[j].x += q.a;
                        if (col + 2 * j + 1 == row) o[j].y += q.a;
                    }
                }
                Q.store(row, col, o);
                if (i == 0 && more) W.store(row, col, o);
                if (i == 0 && !more) to_memory(col, o);
            });
            written();
            if (more) {
                if (!wait_done(0)) break;
                each(0, to_matrix(A));
                written();
            }
            if (i) {
                if (!wait_done(1)) break;
                if (more) each(1, to_matrix(W));
                else each(1, to_memory);
            }
            if (more) {
                if (!wait_done(0)) break;
                each(0, to_matrix(A));
                written();
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) atomicOr(q.status, ERRBIT_TIMEOUT);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 2) tc::tmem_free<1>(tmem, 4 * kRows);
}

// ---------------------------------------------------------------------------
// W X (or X W): a tile of 128 x 128 of the long side a CTA
// ---------------------------------------------------------------------------
struct ApplyControl {
    uint64_t full, done;
    uint32_t tmem;
    int gave_up;
};
constexpr int kApplyStaging = 32 * kChunk * 4;
constexpr int kApplySmem = 1024 + 4 * kMatrix + kEpilogueWarps * kApplyStaging + 64;
static_assert(kApplySmem <= 227 * 1024, "the SM's shared memory");

__global__ void __launch_bounds__(kThreads, 1) short_apply(const __grid_constant__ Short q)
{
    extern __shared__ __align__(1024) unsigned char dynamic[];
    unsigned char* const base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic) + 1023) & ~uintptr_t(1023));
    ApplyControl* const ctl = reinterpret_cast<ApplyControl*>(base + 4 * kMatrix + kEpilogueWarps * kApplyStaging);
    const Matrix W{base, base + kMatrix}, X{base + 2 * kMatrix, base + 3 * kMatrix};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, z = blockIdx.x / q.tiles;
    const int64_t n0 = (int64_t)(blockIdx.x - z * q.tiles) * kRows;
    volatile int* const gave_up = &ctl->gave_up;
    if (threadIdx.x == 0) {
        tc::bar_init(tc::smem_addr(&ctl->full), 1);
        tc::bar_init(tc::smem_addr(&ctl->done), 1);
        ctl->gave_up = 0;
        tc::bar_init_fence();
    }
    if (warp == 2) tc::tmem_alloc<1>(tc::smem_addr(&ctl->tmem), 2 * kRows);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ctl->tmem;
    let_next_begin();
    wait_for_earlier();

    const bool low = q.low_in;
    if (warp == 0 && tc::elect_one()) {
        const uint32_t bar = tc::smem_addr(&ctl->full);
        tc::bar_expect(bar, (low ? 4 : 3) * kMatrix);
        for (int i = 0; i < 2; ++i) {   // 64 of the short side, the products' k
            tc::load_box<1>(tc::smem_addr(W.high) + i * kOperand, &q.w_map, bar, i * kStep, 0, z);
            tc::load_box<1>(tc::smem_addr(W.low) + i * kOperand, &q.w_low_map, bar, i * kStep, 0, z);
            for (int part = 0; part < (low ? 2 : 1); ++part) {
                const CUtensorMap* const map = part ? &q.x_low_apply : &q.x_apply;
                const uint32_t at = tc::smem_addr(part ? X.low : X.high) + i * kOperand;
                if (q.tall) {
                    tc::load_box<1>(at, map, bar, i * kStep, (int)n0, z);
                } else {
                    tc::load_box<1>(at, map, bar, (int)n0, i * kStep, z);
                    tc::load_box<1>(at + kBlockBytes, map, bar, (int)n0 + 64, i * kStep, z);
                }
            }
        }
        if (tc::bar_wait(bar, 0, gave_up)) {
            tc::fence_after();
            for (int i = 0; i < 2; ++i) {
                const uint32_t w = tc::smem_addr(W.high) + i * kOperand, wl = tc::smem_addr(W.low) + i * kOperand;
                const uint32_t x = tc::smem_addr(X.high) + i * kOperand, xl = low ? tc::smem_addr(X.low) + i * kOperand : 0;
                if (q.tall) multiply_split(tmem, x, xl, false, w, wl, false, i == 0);
                else multiply_split(tmem, w, wl, false, x, xl, true, i == 0);
            }
            tc::commit<1>(tc::smem_addr(&ctl->done));
        }
    } else if (warp >= 4 && tc::bar_wait_warp(tc::smem_addr(&ctl->done), 0, gave_up)) {
        tc::fence_after();
        // rows of the accumulator are the short side, or the long one where the matrix is tall
        const int w = warp & 3, c0 = (warp - 4) / 4 * 64, r0 = lane >> 2, p = lane & 3;
        float* const mine = reinterpret_cast<float*>(base + 4 * kMatrix + (warp - 4) * kApplyStaging);
        const float s = q.lift.between(z, q.before, q.before + q.steps) * (q.scale ? q.scale[z] : 1.f);
        const int64_t m_first = (q.tall ? n0 : 0) + w * 32;
        const bool wide = (q.cols & 7) == 0 && (reinterpret_cast<uintptr_t>(q.out) & 15) == 0;
        for (int c = c0; c < c0 + 64; c += kChunk) {
            uint32_t v[32], l[32];
            tc::tmem_load32(tmem + ((uint32_t)(w * 32) << 16) + c, v);
            tc::tmem_load32(tmem + ((uint32_t)(w * 32) << 16) + kRows + c, l);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = s * __fmaf_rn(1.f / kLowScale, __uint_as_float(l[4 * i + j]), __uint_as_float(v[4 * i + j]));
                *reinterpret_cast<float4*>(mine + lane * kChunk + ((i ^ (lane & 7)) * 4)) = make_float4(o[0], o[1], o[2], o[3]);
            }
            __syncwarp();
            const int64_t n = (q.tall ? 0 : n0) + c + p * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i * 8 + r0;
                const int64_t m = m_first + r;
                if (m >= q.rows || n >= q.cols) continue;
                const float4 x = *reinterpret_cast<const float4*>(mine + r * kChunk + (((2 * p) ^ (r & 7)) * 4));
                const float4 y = *reinterpret_cast<const float4*>(mine + r * kChunk + (((2 * p + 1) ^ (r & 7)) * 4));
                const float2 o[4] = {{x.x, x.y}, {x.z, x.w}, {y.x, y.y}, {y.z, y.w}};
                if (q.x_out) {
                    const int64_t at = (z * q.rows + m) * q.ld + n;
                    uint4 high, rest;
                    split8(o, high, rest);
                    *reinterpret_cast<uint4*>(q.x_out + at) = high;
                    *reinterpret_cast<uint4*>(q.x_low_out + at) = rest;
                    continue;
                }
                __nv_bfloat16* const to = q.out + (z * q.rows + m) * q.cols + n;
                if (wide) {
                    *reinterpret_cast<uint4*>(to) = pack8<__nv_bfloat16>(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < q.cols) to[j] = __float2bfloat16_rn(j & 1 ? o[j / 2].y : o[j / 2].x);
                }
            }
            __syncwarp();
        }
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) {   // what was copied lands before the block ends
        atomicOr(q.status, ERRBIT_TIMEOUT);
        const uint64_t t0 = tc::now_ns();
        while (tc::now_ns() - t0 < 2000000) {}
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 2) tc::tmem_free<1>(tmem, 2 * kRows);
}

// Most steps of a pass.
int steps_a_pass(int steps, float a)
{
    const auto until = [&](float growth) {   // W may have grown so much
        const float n = std::log(growth) / std::log(std::fabs(a));
        return !(std::fabs(a) > 1.f) || n > 32.f ? 32 : n < 1.f ? 1 : (int)n;
    };
    return steps <= until(kGrowth) ? steps : until(kGrowthMany);
}

}  // namespace

int run_short(const StepsArgs& p, cudaStream_t st)
{
    const Device dev = device();
    int* const status = dense_status_word();
    if (!dev.sms || !status) return EMB_ERR_CUDA;
    static std::atomic<bool> sized[kMaxDevices];
    if (!sized[dev.number].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(short_steps, cudaFuncAttributeMaxDynamicSharedMemorySize, kStepsSmem) != cudaSuccess ||
            cudaFuncSetAttribute(short_apply, cudaFuncAttributeMaxDynamicSharedMemorySize, kApplySmem) != cudaSuccess) {
            cudaGetLastError();
            return EMB_ERR_CUDA;
        }
        sized[dev.number].store(true, std::memory_order_relaxed);
    }
    Short q;
    q.tall = p.rows > p.cols;
    q.rows = p.rows, q.cols = p.cols, q.ld = p.ld;
    q.w = p.w, q.w_low = p.w_low, q.out = p.out, q.status = status;
    q.a = p.a, q.b = p.b, q.c = p.c;
    q.lift = lift_of(p.lift, p.a, p.steps);
    const int64_t n = q.tall ? p.rows : p.cols, x_elems = p.rows * p.ld;
    q.k_steps = (int)((n + kStep - 1) / kStep);
    q.tiles = (int)((n + kRows - 1) / kRows);
    if (p.batch * q.tiles > INT32_MAX) return EMB_ERR_INVALID_ARG;
    if (!make_map(&q.w_map, EMB_F16, p.w, false, kShort, kShort, p.batch, kShort, kShort * kShort) ||
        !make_map(&q.w_low_map, EMB_F16, p.w_low, false, kShort, kShort, p.batch, kShort, kShort * kShort))
        return EMB_ERR_CUDA;
    const int most = steps_a_pass(p.steps, p.a), passes = (p.steps + most - 1) / most;
    int done = 0;
    for (int i = 0; i < passes; ++i) {
        const int from = i & 1;
        q.low_in = i > 0 || p.low_in;
        q.scale = i > 0 ? nullptr : p.scale;
        q.steps = (p.steps - done + passes - i - 1) / (passes - i);
        q.before = done;
        done += q.steps;
        const bool last = i + 1 == passes;
        q.x_out = last ? nullptr : p.x[from ^ 1];
        q.x_low_out = last ? nullptr : p.x_low[from ^ 1];
        if (!make_map(&q.x, EMB_F16, p.x[from], q.tall, p.cols, p.rows, p.batch, p.ld, x_elems) ||
            !make_map(&q.x_low, EMB_F16, p.x_low[from], q.tall, p.cols, p.rows, p.batch, p.ld, x_elems) ||
            !make_map(&q.x_apply, EMB_F16, p.x[from], !q.tall, p.cols, p.rows, p.batch, p.ld, x_elems) ||
            !make_map(&q.x_low_apply, EMB_F16, p.x_low[from], !q.tall, p.cols, p.rows, p.batch, p.ld, x_elems))
            return EMB_ERR_CUDA;
        if (int rc = launch_next(short_steps, (unsigned)p.batch, kStepsThreads, kStepsSmem, st, 1, q)) return rc;
        if (int rc = launch_next(short_apply, (unsigned)(p.batch * q.tiles), kThreads, kApplySmem, st, 1, q)) return rc;
    }
    return EMB_OK;
}

}  // namespace emb

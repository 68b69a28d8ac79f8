// block_rows of layer norm with a copy that never lands, or with threads whose wait gives up while
// the row's others go on: the kernel as it is, between this file's copies and waits.
#define EMB_NORM_KERNELS
#include "emb_internal.cuh"
#include "rows.cuh"
#include "tensor_core.cuh"

namespace emb {
namespace tc {

__device__ const void* lost_copy;                   // the row of x that is not copied; null: none
__device__ int alone_sub, alone_from, alone_to;     // the threads whose first wait gives up at once

__device__ __forceinline__ void copy_or_lose(uint32_t to, const void* from, uint32_t bytes, uint32_t bar)
{
    if (from != lost_copy) copy_bytes(to, from, bytes, bar);
}

// bar_wait, which ends after 0.2 s
__device__ __forceinline__ bool short_wait(uint32_t bar, uint32_t parity, volatile int* gave_up)
{
    if ((int)threadIdx.y == alone_sub && (int)threadIdx.x >= alone_from && (int)threadIdx.x < alone_to) {
        *gave_up = 1;
        return false;
    }
    const uint64_t start = now_ns();
    while (!bar_try(bar, parity)) {
        if (*gave_up) return false;
        if (now_ns() - start > 200000000) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

}  // namespace tc
}  // namespace emb

#define copy_bytes copy_or_lose
#define bar_wait short_wait
#include "norm.cuh"

using namespace emb;

__global__ void set(const void* lost, int sub, int from, int to)
{
    tc::lost_copy = lost;
    tc::alone_sub = sub, tc::alone_from = from, tc::alone_to = to;
}

// One block over bf16 rows of 1024, `subs` of them at a time (1: the kernel of rows by themselves; with g null the
// forward), row lost's copy left out (-1: none).  status: the call's bits.  The result is CUDA's of the last call.
extern "C" int run(const void* x, const void* g, long rows, void* out, float* dw, float* db, int subs, long lost, int sub, int from, int to, int* status)
{
    constexpr int kWidth = 1024, kTx = 64, kSlot = kWidth * 2;
    const void* const none = lost < 0 ? nullptr : static_cast<const __nv_bfloat16*>(x) + lost * kWidth;
    set<<<1, 1>>>(none, sub, from, to);
    norm::Args a;
    a.x = x, a.g = g, a.x_stride = a.g_stride = kWidth, a.rows = rows, a.width = kWidth, a.eps = 1e-5f;
    a.out = out, a.dw = dw, a.db = db, a.status = status;
    a.stages = 2, a.x_whole = a.g_whole = true, a.x_slot = kSlot, a.g_slot = g ? kSlot : 0;
    const size_t smem = (size_t)subs * a.stages * (a.x_slot + a.g_slot);     // of one row: 8 KB; of more, the sums' 4 KB a row fit as well
    using B = __nv_bfloat16;
    if (!g) norm::block_rows<8, 2, false, false, B, B><<<1, dim3(kTx, 1), smem>>>(a);
    else if (subs == 1) norm::block_rows<8, 2, true, false, B, B><<<1, dim3(kTx, 1), smem>>>(a);
    else norm::block_rows<8, 2, true, true, B, B><<<1, dim3(kTx, subs), smem>>>(a);
    const int rc = (int)cudaGetLastError();
    return rc ? rc : (int)cudaDeviceSynchronize();
}

// Matrix products of the expert layer and of the orthogonalisation (sm_103a):
// what a product computes, shared by its callers and its kernel.
#pragma once

#include "dense_internal.cuh"

namespace emb {

// A number held as fp16 h plus fp16 l / kLowScale: l is h's rounding error, at
// most 2^-11 |h|, scaled up so that it is not lost where h is subnormal.
constexpr float kLowScale = 2048.f;

// D = epilogue(sum_k A[m][k] B[n][k]) over a list of independent problems.  An
// operand is "k-major" when its k runs along memory, "mn-major" when its m (n)
// does.
struct ProductArgs {
    int dtype = EMB_F16;           // of A and B: EMB_F16 or EMB_BF16
    const void* a = nullptr;
    const void* b = nullptr;
    int64_t lda = 0, ldb = 0;      // elements between consecutive rows in memory
    bool a_mn = false, b_mn = false;
    int64_t m = 0, n = 0, k = 0;

    // grouped rows: problem e's rows are [offsets[e], offsets[e + 1]) of P
    //   m_grouped: they are A's and D's m (B is the e-th of a stack)
    //   k_grouped: they are k of A and B (D is the e-th of a stack)
    const int32_t* offsets = nullptr;
    bool m_grouped = false, k_grouped = false;

    // a batch: problem i has its own A, B, C and D, batch strides apart
    int64_t batch = 1, batch_a = 0, batch_b = 0;

    // what follows the sum; every D's and C's row starts at a multiple of 16
    // bytes but a bf16 D's
    //   grouped:             D = sum, in dtype
    //   else, without c:     D = s^2 sum, fp16
    //   with c alone:        D = alpha sum + beta C + diagonal I, fp16
    //   with c and c_low:    D = s (sum + beta (C + C's low part)), fp16 with its low part in d_low, or bf16
    const float* scale = nullptr;  // s of each problem, or null for 1
    float alpha = 1.f, beta = 0.f, diagonal = 0.f;
    const void* c = nullptr;       // laid out as D; fp16
    const void* c_low = nullptr;   // C's scaled rounding error (see kLowScale)
    int64_t ldc = 0, batch_c = 0;
    void* d = nullptr;
    void* d_low = nullptr;
    int d_dtype = EMB_F16;
    int64_t ldd = 0, batch_d = 0;
};

// The same for m-grouped forward products of up to kFewRows rows (few_rows.cu).
constexpr int64_t kFewRows = 4;
int launch_few_rows(const ProductArgs& p, cudaStream_t st);

// Enqueue the product.  EMB_OK or an error with nothing enqueued.
int launch_product(const ProductArgs& p, cudaStream_t st);

}  // namespace emb

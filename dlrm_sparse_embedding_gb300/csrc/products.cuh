// The experts' products (sm_103a): what a product computes, shared by the calls
// and the kernels.
#pragma once

#include "dense_internal.cuh"

namespace emb {

// D[m][n] = sum_k A[m][k] B[n][k] for every group of rows [offsets[e],
// offsets[e + 1]), in 16 bits, every row of every array at a multiple of 16
// bytes.
//   k_grouped false: the rows are m, of A [m][k] and D; B is the e-th weight of a
//                    stack, [n][k] or, with b_mn, [k][n]
//   k_grouped true:  they are k, of A [k][m] and B [k][n]; D is the e-th of a stack
struct ProductArgs {
    int dtype = EMB_F16;           // EMB_F16 or EMB_BF16
    const void* a = nullptr;
    const void* b = nullptr;
    void* d = nullptr;
    int64_t lda = 0, ldb = 0, ldd = 0;   // elements between consecutive rows in memory
    bool b_mn = false, k_grouped = false;
    int64_t m = 0, n = 0, k = 0;   // the grouped one is the number of all rows
    const int32_t* offsets = nullptr;
    int experts = 0;
};

// Forward products of up to kFewRows rows (few_rows.cu).
constexpr int64_t kFewRows = 4;
int launch_few_rows(const ProductArgs& p, cudaStream_t st);

// Enqueue the product.  EMB_OK or an error with nothing enqueued.
int launch_product(const ProductArgs& p, cudaStream_t st);

}  // namespace emb

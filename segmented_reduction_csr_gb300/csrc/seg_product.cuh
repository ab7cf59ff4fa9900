// seg_product.cuh -- matrix products over the rows of offset-delimited
// segments (segments as in GPUSegmentedReduction, "What is an offset-delimited
// segment?"): launch parameters shared by seg_product.cu and api.cu.
//
//   forward   y[r, n]     = sum_k x[r, k] * w[s, k, n]     r in segment s
//   weights   dw[s, k, n] = sum_r x[r, k] * dy[r, n]       over the rows of s
//   adapters  y[r, n]     = sum_k x[r, k] * w[n, k]
//                           + scale[l] * sum_j (sum_k x[r, k] * a[l, j, k]) * b[l, n, j]
//
// All three sum in float32 and round once to the output's type.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace segred {

// Element types of the products (values of seg_dtype_t).
enum : int { PT_F32 = 2, PT_F16 = 3, PT_BF16 = 4 };

struct ProductParams {
    const void* x;          // [R, K], row stride ldx
    const void* w;          // forward: [S][K, N] or [S][N, K] (trans); weights: dy [R, N]
    const void* offsets;    // [S + 1]
    const int32_t* index;   // forward: the matrix of segment s is w[index[s]] (negative: none), or NULL: w[s]
    const float* scale;     // forward with index: the products are scaled by scale[index[s]], or NULL
    void* out;              // forward: [R, N], row stride ldo; weights: [S][K, N]
    int64_t R, K, N, S;
    int64_t ldx, ldw, stride_w, ldo;
    int64_t L;              // forward with index: matrices in w
    int32_t off64, trans, type, out_type;
    // adapters: the low-rank part added to the shared product
    const float* u;         // [R, rank] scaled products with a
    const void* b;          // [L][N, rank]
    int64_t rank;
};

cudaError_t launch_product(const ProductParams& p, cudaStream_t stream);
cudaError_t launch_product_grad(const ProductParams& p, cudaStream_t stream);
cudaError_t launch_lora(const ProductParams& p, cudaStream_t stream);

}  // namespace segred

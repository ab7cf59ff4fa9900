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
    const void* w;          // forward: [S][K, N] or [S][N, K] (trans); weights: dy [R, N]; adapters: [N, K]
    const void* offsets;    // [S + 1]
    const int32_t* index;   // forward: the matrix of segment s is w[index[s]] (outside [0, L): none), or NULL: w[s]
    const float* scale;     // forward with index: products are scaled by scale[index[s]], or NULL
    void* out;              // forward: [R, N], row stride ldo; weights: [S][K, N]
    int64_t R, K, N, S;
    int64_t ldx, ldw, stride_w, ldo;
    int64_t L;              // matrices that index names
    int32_t off64, trans, type, out_type;
    // adapters: the low-rank part added to the shared product
    const float* u;         // [R, rank] scaled products with a
    const void* b;          // [L][N, rank]
    int64_t rank;
    int32_t overlap;        // u's kernel lets this one start beside it
    // library-owned
    unsigned char* ws;      // see ProductPlan
    unsigned int* status;   // device status word
    int32_t sms;
};

// How a call is launched; a pure function of sizes, strides, alignment and the SM count.
struct ProductPlan {
    int32_t grid;
    int32_t too_many;       // 1: more tiles than 31 bits count
    int32_t tensor;         // 1: operands come by tensor copies, 0: by the loader warps
    int32_t narrow;         // 1: at most 64 rows per tile and a deeper ring (always without tensor copies)
    int32_t pair;           // 1: two CTAs share a tile
    int32_t empty;          // 1: no sum has a term
    int32_t pack_x, pack_w; // 1: the operand is first laid out in 16-byte aligned rows
    int32_t mtiles, ntiles; // tiles of the output's contiguous / other dimension (forward: rows vary by segment)
    int32_t parts;          // forward: parts of the contraction
    int32_t part_blocks;    // forward: 64-wide blocks per part
    int64_t chunk;          // weights: rows per part of a segment
    int32_t add_blocks;     // weights: blocks of the kernel that adds the parts (0: no segment can be split)
    int32_t add_by_start;   // weights: those blocks stand for `chunk` rows each, not for a segment each
    int32_t staged;         // forward, adapters: the sums are kept in float32 scratch and rounded by a kernel of their own
    int64_t row_tiles;      // forward: most row tiles there can be
    int64_t prefix_bytes, partial_bytes, staged_bytes, pack_x_bytes, pack_w_bytes;   // the workspace, in this order
    int64_t bytes() const { return prefix_bytes + partial_bytes + staged_bytes + pack_x_bytes + pack_w_bytes; }
};

enum : int { PRODUCT_FORWARD = 0, PRODUCT_WEIGHTS = 1, PRODUCT_ADAPTERS = 2 };

ProductPlan plan_product(int mode, const ProductParams& p);
// Columns of the tile that `plan` counts in and that is launched for it.
int product_tile_columns(const ProductParams& p, const ProductPlan& plan);
cudaError_t launch_product(int mode, const ProductParams& p, const ProductPlan& plan, cudaStream_t stream);

// u of the adapters (forward with index, rank columns, float32 result) for
// calls with a few rows per segment at most.
bool lora_by_rows(const ProductParams& p);
cudaError_t launch_lora_rows(const ProductParams& p, cudaStream_t stream);

}  // namespace segred

// seg_norm.cuh -- layer norm of the rows of offset-delimited segments, with a
// weight and bias for every segment: launch parameters shared by seg_norm.cu
// and api.cu.
//
//   forward   z = (x - mean) * rstd,  y = z * w + b       mean, rstd of the row
//   backward  g = dy * w,  dx = rstd * (g - sum(g) / F - z * sum(g z) / F)
//             dw[s] = sum_r dy * z,  db[s] = sum_r dy     over the rows of s
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace segred {

struct NormParams {
    const void* x;          // [R, F], row stride ldx
    const void* dy;         // backward: [R, F], row stride ldy
    const void* weight;     // [S, F] (offsets NULL: [F]), or NULL for 1
    const void* bias;       // the same, or NULL for 0
    const void* offsets;    // [S + 1], or NULL: one segment of all rows (S = 1)
    void* out;              // y, or dx (NULL: not wanted); row stride ldo
    float* mean;            // [R]: written (or NULL), or given
    float* rstd;
    void* dweight;          // [S, F] of weight_type, or NULL
    void* dbias;
    int64_t R, F, S;
    int64_t ldx, ldy, ldo;
    float eps;
    int32_t type, weight_type, off64;      // PT_F32, PT_F16 or PT_BF16
    // library-owned
    unsigned char* ws;      // see NormPlan
    int32_t sms;
};

// How a call is launched; a pure function of sizes, strides, alignment and the SM count.
struct NormPlan {
    int32_t aligned;        // 1: rows and weights are whole 16-byte units
    int32_t per;            // such units that a thread has of a row, 0: rows are read again instead of kept
    int32_t group;          // threads of a row, a power of two
    int32_t threads;        // of a block
    int64_t chunk, chunks;  // rows of a block; blocks
    int32_t tiles;          // backward: tiles of columns, each with blocks of its own
    int32_t clear_blocks;   // backward: blocks of the kernel that clears the sums of segments without rows (0: the others do)
    int64_t sums_bytes, partial_bytes;     // each row's two sums, where tiles share them; the parts of the column sums
    // The workspace of a call, in this order: the rows' sums are for dx, the parts for the others.
    int64_t sums_for(const NormParams& p) const { return p.out ? sums_bytes : 0; }
    int64_t parts_for(const NormParams& p) const { return p.dweight || p.dbias ? partial_bytes : 0; }
};

NormPlan plan_norm(bool grad, const NormParams& p);
cudaError_t launch_norm(const NormParams& p, const NormPlan& plan, cudaStream_t stream);
cudaError_t launch_norm_grad(const NormParams& p, const NormPlan& plan, cudaStream_t stream);

}  // namespace segred

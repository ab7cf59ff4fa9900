// seg_gated.cuh -- the gated feed-forward block's activation and its gradient
// over rows of products that are there already: launch parameters shared by
// seg_gated.cu and api.cu.  (seg_product.cu has the kernel that applies it to
// the products as they are summed.)
//
//   forward   out = act(g) * u                  g, u: the halves of a row of pre
//   backward  dg = dy * u * act'(g),  du = dy * act(g)
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace segred {

// seg_activation_t
enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3, ACT_SIGMOID = 4 };

struct GatedParams {
    const void* pre;        // [R, 2 N], row stride ldp; forward: float32, backward: of pre_type
    const void* dy;         // backward: [R, N], row stride ldy
    void* out;              // forward: [R, N], backward: [R, 2 N]; row stride ldo
    void* rounded;          // forward: pre in `type` [R, 2 N], row stride ldr, or NULL
    int64_t R, N;
    int64_t ldp, ldy, ldo, ldr;
    int32_t type, pre_type, activation;    // pre_type: PT_F32, or type
    int32_t sms;
};

cudaError_t launch_gated(const GatedParams& p, cudaStream_t stream);
cudaError_t launch_gated_grad(const GatedParams& p, cudaStream_t stream);

}  // namespace segred

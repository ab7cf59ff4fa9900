// seg_gated.cu -- the gated block's activation over rows in memory (see
// seg_gated.cuh): one pass, 16 bytes of each half of a row per thread where the
// rows allow it.  Bound by memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "seg_act.cuh"
#include "seg_product.cuh"

namespace segred {
namespace {

template <class T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T, int V> struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Pack {
    T v[V];
};

// `lanes` threads a row, V columns of it each at a time.
template <class T, class P, int V, bool GRAD>
__global__ void __launch_bounds__(256) gated_kernel(const __grid_constant__ GatedParams p, int lanes) {
    constexpr bool FAST = sizeof(T) == 2;
    const int lane = threadIdx.x % lanes;
    const int64_t step = int64_t(gridDim.x) * (256 / lanes);
    for (int64_t r = int64_t(blockIdx.x) * (256 / lanes) + threadIdx.x / lanes; r < p.R; r += step) {
        for (int64_t c = int64_t(lane) * V; c < p.N; c += lanes * V) {
            if constexpr (GRAD) {
                const P* pre = static_cast<const P*>(p.pre) + r * p.ldp + c;
                const Pack<P, V> g = *reinterpret_cast<const Pack<P, V>*>(pre), u = *reinterpret_cast<const Pack<P, V>*>(pre + p.N);
                const Pack<T, V> dy = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p.dy) + r * p.ldy + c);
                Pack<T, V> dg, du;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float slope;
                    const float f = activate<FAST, true>(p.activation, to_float<P>(g.v[i]), slope), d = to_float<T>(dy.v[i]);
                    dg.v[i] = from_float<T>(d * to_float<P>(u.v[i]) * slope);
                    du.v[i] = from_float<T>(d * f);
                }
                T* out = static_cast<T*>(p.out) + r * p.ldo + c;
                *reinterpret_cast<Pack<T, V>*>(out) = dg;
                *reinterpret_cast<Pack<T, V>*>(out + p.N) = du;
            } else {
                const float* pre = static_cast<const float*>(p.pre) + r * p.ldp + c;
                const Pack<float, V> g = *reinterpret_cast<const Pack<float, V>*>(pre), u = *reinterpret_cast<const Pack<float, V>*>(pre + p.N);
                Pack<T, V> o, rg, ru;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float slope;
                    o.v[i] = from_float<T>(activate<FAST, false>(p.activation, g.v[i], slope) * u.v[i]);
                    rg.v[i] = from_float<T>(g.v[i]);
                    ru.v[i] = from_float<T>(u.v[i]);
                }
                *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.out) + r * p.ldo + c) = o;
                if (p.rounded) {
                    T* rounded = static_cast<T*>(p.rounded) + r * p.ldr + c;
                    *reinterpret_cast<Pack<T, V>*>(rounded) = rg;
                    *reinterpret_cast<Pack<T, V>*>(rounded + p.N) = ru;
                }
            }
        }
    }
}

bool fits(const void* ptr, int64_t ld, int size) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld * size % 16 == 0; }

template <class T, class P, bool GRAD>
cudaError_t launch(const GatedParams& p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = p.N % V == 0 && fits(p.pre, p.ldp, sizeof(P)) && fits(p.out, p.ldo, sizeof(T)) &&
                     (!GRAD || fits(p.dy, p.ldy, sizeof(T))) && (!p.rounded || fits(p.rounded, p.ldr, sizeof(T)));
    int lanes = 4;
    while (lanes < 256 && lanes * (vec ? V : 1) < p.N) lanes *= 2;
    const int rows = 256 / lanes;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((p.R + rows - 1) / rows, int64_t(p.sms) * 32));
    if (vec) gated_kernel<T, P, V, GRAD><<<blocks, 256, 0, stream>>>(p, lanes);
    else gated_kernel<T, P, 1, GRAD><<<blocks, 256, 0, stream>>>(p, lanes);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated(const GatedParams& p, cudaStream_t stream) {
    if (p.type == PT_F32) return launch<float, float, false>(p, stream);
    if (p.type == PT_F16) return launch<__half, float, false>(p, stream);
    return launch<__nv_bfloat16, float, false>(p, stream);
}

cudaError_t launch_gated_grad(const GatedParams& p, cudaStream_t stream) {
    const bool wide = p.pre_type == PT_F32;
    if (p.type == PT_F32) return launch<float, float, true>(p, stream);
    if (p.type == PT_F16) return wide ? launch<__half, float, true>(p, stream) : launch<__half, __half, true>(p, stream);
    return wide ? launch<__nv_bfloat16, float, true>(p, stream) : launch<__nv_bfloat16, __nv_bfloat16, true>(p, stream);
}

}  // namespace segred

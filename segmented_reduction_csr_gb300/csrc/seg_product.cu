// seg_product.cu -- products over the rows of segments (see seg_product.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "seg_product.cuh"

namespace segred {
namespace {

constexpr int PT = 64;    // output tile side
constexpr int PK = 16;    // contraction step

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ int64_t offset_at(const ProductParams& p, int64_t s) {
    int64_t o = p.off64 ? __ldg(static_cast<const int64_t*>(p.offsets) + s)
                        : static_cast<int64_t>(__ldg(static_cast<const uint32_t*>(p.offsets) + s));
    o = o < 0 ? 0 : o;
    return o > p.R ? p.R : o;
}

// acc[i][j] += sum_k A(m0 + 4 ty + i, k) * B(k, n0 + 4 tx + j) for k < kn
template <class FA, class FB>
__device__ __forceinline__ void tile_product(FA fa, FB fb, int64_t kn, float (&acc)[4][4]) {
    __shared__ float as[PK][PT + 4], bs[PK][PT + 4];
    const int t = threadIdx.x, tx = t % 16, ty = t / 16;
    for (int64_t k0 = 0; k0 < kn; k0 += PK) {
        for (int i = t; i < PK * PT; i += 256) {
            as[i / PT][i % PT] = k0 + i / PT < kn ? fa(i % PT, k0 + i / PT) : 0.0f;
            bs[i / PT][i % PT] = k0 + i / PT < kn ? fb(i % PT, k0 + i / PT) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < PK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += as[k][4 * ty + i] * bs[k][4 * tx + j];
        __syncthreads();
    }
}

// One CTA per (64 columns of the output, segment); row S is the rows in no segment.
template <class T, class TO>
__global__ void __launch_bounds__(256) forward_kernel(ProductParams p) {
    const int64_t n0 = int64_t(blockIdx.x) * PT;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const T* x = static_cast<const T*>(p.x);
    TO* out = static_cast<TO*>(p.out);
    for (int64_t s = blockIdx.y; s <= p.S; s += gridDim.y) {
        if (s == p.S) {
            const int64_t b = p.S > 0 ? offset_at(p, 0) : 0, e = p.S > 0 ? offset_at(p, p.S) : 0;
            for (int64_t i = threadIdx.x; i < p.R * PT; i += 256) {
                const int64_t r = i / PT, n = n0 + i % PT;
                if ((r < b || r >= e) && n < p.N) out[r * p.ldo + n] = from_f<TO>(0.0f);
            }
            continue;
        }
        const int64_t b = offset_at(p, s), e = offset_at(p, s + 1);
        const int64_t m = p.index ? __ldg(p.index + s) : s;
        const bool have = !p.index || (m >= 0 && m < p.L);
        const T* w = static_cast<const T*>(p.w) + (have ? m : 0) * p.stride_w;
        const float sc = have && p.scale ? __ldg(p.scale + m) : 1.0f;
        for (int64_t r0 = b; r0 < e; r0 += PT) {
            float acc[4][4] = {};
            tile_product([&](int i, int64_t k) { return r0 + i < e ? to_f(x[(r0 + i) * p.ldx + k]) : 0.0f; },
                         [&](int j, int64_t k) {
                             return n0 + j < p.N ? to_f(p.trans ? w[(n0 + j) * p.ldw + k] : w[k * p.ldw + n0 + j]) : 0.0f;
                         },
                         have ? p.K : 0, acc);
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int64_t r = r0 + 4 * ty + i, n = n0 + 4 * tx + j;
                    if (r < e && n < p.N) out[r * p.ldo + n] = from_f<TO>(acc[i][j] * sc);
                }
        }
    }
}

// One CTA per (64 x 64 tile of dw, segment).
template <class T, class TO>
__global__ void __launch_bounds__(256) grad_kernel(ProductParams p) {
    const int64_t n0 = int64_t(blockIdx.x) * PT, k0 = int64_t(blockIdx.y) * PT;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.w);
    for (int64_t s = blockIdx.z; s < p.S; s += gridDim.z) {
        const int64_t b = offset_at(p, s), e = offset_at(p, s + 1);
        float acc[4][4] = {};
        tile_product([&](int i, int64_t r) { return k0 + i < p.K ? to_f(x[(b + r) * p.ldx + k0 + i]) : 0.0f; },
                     [&](int j, int64_t r) { return n0 + j < p.N ? to_f(dy[(b + r) * p.ldw + n0 + j]) : 0.0f; },
                     e > b ? e - b : 0, acc);
        TO* out = static_cast<TO*>(p.out) + s * p.K * p.N;
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t k = k0 + 4 * ty + i, n = n0 + 4 * tx + j;
                if (k < p.K && n < p.N) out[k * p.N + n] = from_f<TO>(acc[i][j]);
            }
    }
}

// The shared product and the low-rank part: one CTA per 64 x 64 tile of the output.
template <class T>
__global__ void __launch_bounds__(256) lora_kernel(ProductParams p) {
    const int64_t n0 = int64_t(blockIdx.x) * PT;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const T* x = static_cast<const T*>(p.x);
    const T* w = static_cast<const T*>(p.w);
    T* out = static_cast<T*>(p.out);
    for (int64_t r0 = int64_t(blockIdx.y) * PT; r0 < p.R; r0 += int64_t(gridDim.y) * PT) {
        float acc[4][4] = {};
        tile_product([&](int i, int64_t k) { return r0 + i < p.R ? to_f(x[(r0 + i) * p.ldx + k]) : 0.0f; },
                     [&](int j, int64_t k) { return n0 + j < p.N ? to_f(w[(n0 + j) * p.ldw + k]) : 0.0f; }, p.K, acc);
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 4 * ty + i;
            if (r >= p.R) continue;
            int64_t lo = 0, hi = p.S;   // the last segment that starts at or before r
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (offset_at(p, mid) <= r) lo = mid; else hi = mid;
            }
            int64_t l = -1;
            if (p.S > 0 && offset_at(p, lo) <= r && r < offset_at(p, lo + 1)) l = __ldg(p.index + lo);
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + 4 * tx + j;
                if (n >= p.N) continue;
                float v = acc[i][j];
                if (l >= 0 && l < p.L)
                    for (int64_t q = 0; q < p.rank; ++q)
                        v += p.u[r * p.rank + q] * to_f(static_cast<const T*>(p.b)[(l * p.N + n) * p.rank + q]);
                out[r * p.ldo + n] = from_f<T>(v);
            }
        }
    }
}

template <class F>
cudaError_t by_type(int type, F f) {
    if (type == PT_F32) return f(float());
    if (type == PT_F16) return f(__half());
    return f(__nv_bfloat16());
}

unsigned tiles(int64_t n, int64_t most = 65535) {
    const int64_t t = (n + PT - 1) / PT;
    return static_cast<unsigned>(t < most ? (t < 1 ? 1 : t) : most);
}

}  // namespace

cudaError_t launch_product(const ProductParams& p, cudaStream_t stream) {
    return by_type(p.type, [&](auto t) {
        using T = decltype(t);
        const dim3 grid(tiles(p.N, 1 << 30), static_cast<unsigned>(p.S < 65000 ? p.S + 1 : 65000));
        if (p.out_type == PT_F32) forward_kernel<T, float><<<grid, 256, 0, stream>>>(p);
        else forward_kernel<T, T><<<grid, 256, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_product_grad(const ProductParams& p, cudaStream_t stream) {
    return by_type(p.type, [&](auto t) {
        using T = decltype(t);
        const dim3 grid(tiles(p.N, 1 << 30), tiles(p.K), static_cast<unsigned>(p.S < 65000 ? p.S : 65000));
        if (p.out_type == PT_F32) grad_kernel<T, float><<<grid, 256, 0, stream>>>(p);
        else grad_kernel<T, T><<<grid, 256, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_lora(const ProductParams& p, cudaStream_t stream) {
    return by_type(p.type, [&](auto t) {
        using T = decltype(t);
        lora_kernel<T><<<dim3(tiles(p.N, 1 << 30), tiles(p.R)), 256, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace segred

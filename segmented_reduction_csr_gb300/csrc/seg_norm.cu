// seg_norm.cu -- layer norm of the rows of segments (see seg_norm.cuh).
//
// A group of threads has a row, in registers: one read of it serves the mean,
// then the centred squares (no difference of large sums), then the result.
// Groups of up to 32 threads add with shuffles, larger ones through shared
// memory and a barrier of their own.  Everything is float32 and rounded once.
//
// Backward: a block has a chunk of neighbouring rows and takes the runs of rows
// of one segment in it one after the other.  A thread keeps its columns' sums
// of dy z and dy in registers over a run; the block's groups are added at its
// end.  A segment that lies in one chunk gets its sums there; of the others
// every chunk stores a part, and a second kernel adds a segment's parts in the
// order of the chunks, so results repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "seg_common.cuh"
#include "seg_norm.cuh"
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

// V values that are loaded and stored together.
template <class T, int V> struct alignas(V * sizeof(T)) Pack {
    T v[V];
};
template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
    if constexpr (V * sizeof(T) == 16) {
        union {
            uint4 u;
            Pack<T, V> x;
        } r = {__ldg(reinterpret_cast<const uint4*>(p))};
        return r.x;
    } else {
        return *reinterpret_cast<const Pack<T, V>*>(p);
    }
}

// V neighbouring values of weight_type at element `at`.
template <class T, int V>
__device__ __forceinline__ void load_weights(const void* w, bool wide, int64_t at, float (&f)[V]) {
    if (wide) {
        const float* p = static_cast<const float*>(w) + at;
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p + i));
                f[i] = x.x, f[i + 1] = x.y, f[i + 2] = x.z, f[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
        }
    } else {
        const Pack<T, V> x = load_pack<T, V>(static_cast<const T*>(w) + at);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_float<T>(x.v[i]);
    }
}

__device__ __forceinline__ int64_t offset_at(const NormParams& p, int64_t s) {
    const int64_t o = p.off64 ? __ldg(static_cast<const int64_t*>(p.offsets) + s)
                              : static_cast<int64_t>(__ldg(static_cast<const uint32_t*>(p.offsets) + s));
    return clamp_off(o, p.R);
}

// The run of rows that row r is in: its segment s (-1: none) and where it begins and ends.
struct Run {
    int64_t s = -1, begin = 0, end = 0;
};
__device__ __forceinline__ Run run_of(const NormParams& p, int64_t r) {
    if (!p.offsets) return {0, 0, p.R};
    int64_t lo = -1, hi = p.S;      // the last offset at or before r; hi: the first one after it, or S
    if (p.S > 0 && offset_at(p, p.S) <= r) lo = p.S;
    else
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (offset_at(p, mid) <= r) lo = mid; else hi = mid;
        }
    Run x;
    if (lo < 0 || lo >= p.S) {
        x.begin = lo < 0 ? 0 : r;
        x.end = lo < 0 && p.S > 0 ? offset_at(p, 0) : p.R;
    } else {
        x.s = lo;
        x.begin = offset_at(p, lo);
        x.end = offset_at(p, lo + 1);
    }
    if (x.end <= r) x.s = -1, x.end = r + 1;      // (offsets that decrease: the next row may be found)
    return x;
}

// Sums of N values over a row's threads, to all of them.  `red`: [2][8 or 16 warps][N], used in turns.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int group, float* red, int& turn) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        if (d < group) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
        }
    }
    if (group > 32) {
        const int warps = group >> 5, warp = threadIdx.x >> 5, first = warp / warps * warps;
        float* at = red + turn * (blockDim.x >> 5) * N;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) at[warp * N + i] = v[i];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / warps), "r"(group) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += at[(first + w) * N + i];
        turn ^= 1;
    }
}

// ---------------------------------------------------------------------------

template <class T, int V, int PER>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ NormParams p, int group, int64_t chunk) {
    __shared__ float red[2 * 8];
    const int t = threadIdx.x % group, g = threadIdx.x / group, groups = 256 / group;
    const int64_t c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, p.R);
    const float inv = 1.0f / static_cast<float>(p.F);
    const bool wide = p.weight_type == PT_F32;
    int turn = 0;
    Run run;
    for (int64_t base = c0; base < c1; base += groups) {
        const int64_t r = base + g;
        const bool in = r < c1;
        const T* x = static_cast<const T*>(p.x) + (in ? r : c0) * p.ldx;
        Pack<T, V> raw[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int64_t c = (int64_t(j) * group + t) * V;
            if (c < p.F) raw[j] = load_pack<T, V>(x + c);
        }
        if (in && r >= run.end) run = run_of(p, r);
        float sum[1] = {0.0f}, sq[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if ((int64_t(j) * group + t) * V < p.F)
#pragma unroll
                for (int i = 0; i < V; ++i) sum[0] += to_float<T>(raw[j].v[i]);
        }
        group_sum<1>(sum, group, red, turn);
        const float mean = sum[0] * inv;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if ((int64_t(j) * group + t) * V < p.F)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = to_float<T>(raw[j].v[i]) - mean;
                    sq[0] = fmaf(d, d, sq[0]);
                }
        }
        group_sum<1>(sq, group, red, turn);
        const float rstd = 1.0f / sqrtf(fmaf(sq[0], inv, p.eps));
        if (!in) continue;
        const bool used = run.s >= 0;
        if (t == 0) {
            if (p.mean) p.mean[r] = used ? mean : 0.0f;
            if (p.rstd) p.rstd[r] = used ? rstd : 0.0f;
        }
        T* y = static_cast<T*>(p.out) + r * p.ldo;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int64_t c = (int64_t(j) * group + t) * V;
            if (c >= p.F) continue;
            float w[V], b[V];
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = 1.0f, b[i] = 0.0f;
            if (used && p.weight) load_weights<T, V>(p.weight, wide, run.s * p.F + c, w);
            if (used && p.bias) load_weights<T, V>(p.bias, wide, run.s * p.F + c, b);
            Pack<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float z = (to_float<T>(raw[j].v[i]) - mean) * rstd;
                o.v[i] = from_float<T>(used ? fmaf(z, w[i], b[i]) : 0.0f);
            }
            *reinterpret_cast<Pack<T, V>*>(y + c) = o;
        }
    }
}

// Sum of one value over the block (256 threads), to all of them.
__device__ __forceinline__ float block_sum(float v, float* red) {
    float x[1] = {v};
    int turn = 0;
    __syncthreads();
    group_sum<1>(x, 256, red, turn);
    return x[0];
}

// Rows of more columns than a block's registers hold: read three times, the
// second and third from L2.
template <class T>
__global__ void __launch_bounds__(256) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[2 * 8];
    const float inv = 1.0f / static_cast<float>(p.F);
    const bool wide = p.weight_type == PT_F32;
    Run run;
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        if (r >= run.end) run = run_of(p, r);
        float sum = 0.0f, sq = 0.0f;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) sum += to_float<T>(x[c]);
        const float mean = block_sum(sum, red) * inv;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) {
            const float d = to_float<T>(x[c]) - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = 1.0f / sqrtf(fmaf(block_sum(sq, red), inv, p.eps));
        const bool used = run.s >= 0;
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = used ? mean : 0.0f;
            if (p.rstd) p.rstd[r] = used ? rstd : 0.0f;
        }
        T* y = static_cast<T*>(p.out) + r * p.ldo;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) {
            float w[1] = {1.0f}, b[1] = {0.0f};
            if (used && p.weight) load_weights<T, 1>(p.weight, wide, run.s * p.F + c, w);
            if (used && p.bias) load_weights<T, 1>(p.bias, wide, run.s * p.F + c, b);
            y[c] = from_float<T>(used ? fmaf((to_float<T>(x[c]) - mean) * rstd, w[0], b[0]) : 0.0f);
        }
    }
}

// ---------------------------------------------------------------------------

struct GradArgs {
    NormParams p;
    int32_t group, tile;        // columns of a tile
    int64_t chunk;
    float* sums;                // [R][2]: sum(g), sum(g z) of each row, or NULL: a block has all columns
    float* partials;            // [2 chunks][2][F]: the first and last run of a chunk
};

// The two sums of each row, where a block does not have all its columns.
template <class T>
__global__ void __launch_bounds__(256) norm_sums_kernel(const __grid_constant__ GradArgs a) {
    __shared__ float red[2 * 8];
    const NormParams& p = a.p;
    const bool wide = p.weight_type == PT_F32;
    Run run;
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
        if (r >= run.end) run = run_of(p, r);
        if (run.s < 0) continue;
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        const T* dy = static_cast<const T*>(p.dy) + r * p.ldy;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) {
            float w[1] = {1.0f};
            if (p.weight) load_weights<T, 1>(p.weight, wide, run.s * p.F + c, w);
            const float gr = to_float<T>(dy[c]) * w[0];
            s1 += gr;
            s2 = fmaf(gr, (to_float<T>(x[c]) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, red);
        s2 = block_sum(s2, red);
        if (threadIdx.x == 0) a.sums[2 * r] = s1, a.sums[2 * r + 1] = s2;
    }
}

__device__ __forceinline__ void store_weight(void* out, int type, int64_t at, float v) {
    if (type == PT_F32) static_cast<float*>(out)[at] = v;
    else if (type == PT_F16) static_cast<__half*>(out)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

template <class T, int V, int PER, int NT>
__global__ void __launch_bounds__(NT) norm_grad_kernel(const __grid_constant__ GradArgs a) {
    constexpr int E = V * PER;
    __shared__ float red[2 * NT / 32 * 2];
    extern __shared__ float shared_sums[];       // [groups of at least a warp][2][tile]
    const NormParams& p = a.p;
    const int group = a.group, t = threadIdx.x % group, g = threadIdx.x / group, groups = NT / group;
    const int64_t c0 = blockIdx.x * a.chunk, c1 = min(c0 + a.chunk, p.R);
    const int64_t col0 = int64_t(blockIdx.y) * a.tile;
    const float inv = 1.0f / static_cast<float>(p.F);
    const bool wide = p.weight_type == PT_F32, want_dx = p.out != nullptr, want_dw = p.dweight || p.dbias;
    auto column = [&](int j) { return col0 + (int64_t(j) * group + t) * V; };
    int turn = 0;
    if (want_dw && p.offsets) {
        // segments without rows
        const int64_t each = (p.S + gridDim.x - 1) / gridDim.x, s1 = min((blockIdx.x + 1) * each, p.S);
        for (int64_t s = blockIdx.x * each; s < s1; ++s) {
            if (offset_at(p, s) < offset_at(p, s + 1)) continue;
            for (int64_t c = col0 + threadIdx.x; c < min(col0 + a.tile, p.F); c += NT) {
                if (p.dweight) store_weight(p.dweight, p.weight_type, s * p.F + c, 0.0f);
                if (p.dbias) store_weight(p.dbias, p.weight_type, s * p.F + c, 0.0f);
            }
        }
    }
    for (int64_t r0 = c0; r0 < c1;) {
        const Run run = run_of(p, r0);
        const int64_t r1 = min(run.end, c1);
        if (run.s < 0) {
            // rows in no segment
            if (want_dx)
                for (int64_t r = r0 + g; r < r1; r += groups)
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        Pack<T, V> zero;
#pragma unroll
                        for (int i = 0; i < V; ++i) zero.v[i] = from_float<T>(0.0f);
                        if (column(j) < p.F) *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.out) + r * p.ldo + column(j)) = zero;
                    }
            r0 = r1;
            continue;
        }
        float w[PER][V], dw[E], db[E];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[j][i] = 1.0f, dw[j * V + i] = 0.0f, db[j * V + i] = 0.0f;
            if (p.weight && column(j) < p.F) load_weights<T, V>(p.weight, wide, run.s * p.F + column(j), w[j]);
        }
        for (int64_t base = r0; base < r1; base += groups) {
            const int64_t r = base + g;
            const bool in = r < r1;
            Pack<T, V> x[PER], dy[PER];
            float mean = 0.0f, rstd = 0.0f;
            if (in) {
                const T* px = static_cast<const T*>(p.x) + r * p.ldx;
                const T* pd = static_cast<const T*>(p.dy) + r * p.ldy;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (column(j) < p.F) x[j] = load_pack<T, V>(px + column(j)), dy[j] = load_pack<T, V>(pd + column(j));
                }
                mean = __ldg(p.mean + r);
                rstd = __ldg(p.rstd + r);
            }
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (!in || column(j) >= p.F) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = to_float<T>(dy[j].v[i]), z = (to_float<T>(x[j].v[i]) - mean) * rstd, gr = d * w[j][i];
                    db[j * V + i] += d;
                    dw[j * V + i] = fmaf(d, z, dw[j * V + i]);
                    s[0] += gr;
                    s[1] = fmaf(gr, z, s[1]);
                }
            }
            if (!want_dx) continue;
            if (!a.sums) group_sum<2>(s, group, red, turn);
            else if (in) s[0] = __ldg(a.sums + 2 * r), s[1] = __ldg(a.sums + 2 * r + 1);
            if (!in) continue;
            const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (column(j) >= p.F) continue;
                Pack<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float z = (to_float<T>(x[j].v[i]) - mean) * rstd;
                    o.v[i] = from_float<T>(rstd * (fmaf(to_float<T>(dy[j].v[i]), w[j][i], -m1) - z * m2));
                }
                *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.out) + r * p.ldo + column(j)) = o;
            }
        }
        if (want_dw) {
            // the groups' sums, in their order: of a warp's groups first, then of the warps
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                if (d < group) continue;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], d);
                    db[i] += __shfl_xor_sync(0xffffffffu, db[i], d);
                }
            }
            const int wide_group = max(group, 32), parts = NT / wide_group, part = threadIdx.x / wide_group;
            __syncthreads();
            if (threadIdx.x % wide_group < group) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int c = (j * group + t) * V + i;
                        if (c >= a.tile) continue;
                        shared_sums[(part * 2) * a.tile + c] = dw[j * V + i];
                        shared_sums[(part * 2 + 1) * a.tile + c] = db[j * V + i];
                    }
            }
            __syncthreads();
            const bool whole = run.begin >= c0 && run.end <= c1;
            float* slot = a.partials + (2 * int64_t(blockIdx.x) + (run.begin >= c0 ? 1 : 0)) * 2 * p.F;
            for (int i = threadIdx.x; i < 2 * a.tile; i += NT) {
                const int which = i >= a.tile;
                const int64_t c = col0 + i - which * a.tile;
                if (c >= p.F) continue;
                float v = 0.0f;
                for (int q = 0; q < parts; ++q) v += shared_sums[q * 2 * a.tile + i];
                void* out = which ? p.dbias : p.dweight;
                if (!whole) slot[which * p.F + c] = v;
                else if (out) store_weight(out, p.weight_type, run.s * p.F + c, v);
            }
        }
        r0 = r1;
    }
}

// Adds the parts of a segment that more than one chunk has rows of: blockIdx.x
// names the segment, or (by_start) the chunk in which it starts; blockIdx.y the
// first 32 of the 2 F sums.  Each warp adds an equal share of the parts in order, then
// the warps' sums are added.
__global__ void __launch_bounds__(256) norm_add_kernel(const __grid_constant__ GradArgs a, int by_start) {
    __shared__ float sums[8][32];
    const NormParams& p = a.p;
    int64_t s = blockIdx.x, begin = 0, end = p.R;
    if (by_start) {
        const Run run = run_of(p, min((int64_t(blockIdx.x) + 1) * a.chunk, p.R) - 1);
        s = run.s, begin = run.begin, end = run.end;
        if (s < 0 || begin / a.chunk != blockIdx.x) return;
    } else if (p.offsets) {
        begin = offset_at(p, s), end = offset_at(p, s + 1);
    }
    if (begin >= end) return;
    const int64_t first = begin / a.chunk, last = (end - 1) / a.chunk;
    if (first == last) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t parts = last - first + 1, each = (parts + 7) / 8;
    const int64_t q0 = warp * each, q1 = min(q0 + each, parts);
    for (int64_t i0 = int64_t(blockIdx.y) * 32; i0 < 2 * p.F; i0 += int64_t(gridDim.y) * 32) {
        const int64_t i = i0 + lane;
        float v = 0.0f;
        if (i < 2 * p.F) {
#pragma unroll 8
            for (int64_t q = q0; q < q1; ++q) v += __ldcg(a.partials + (2 * (first + q) + (q == 0 ? 1 : 0)) * 2 * p.F + i);
        }
        sums[warp][lane] = v;
        __syncthreads();
        if (warp == 0 && i < 2 * p.F) {
            v = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) v += sums[q][lane];
            void* out = i < p.F ? p.dweight : p.dbias;
            if (out) store_weight(out, p.weight_type, s * p.F + (i < p.F ? i : i - p.F), v);
        }
        __syncthreads();
    }
}

int64_t ceil_to(int64_t n, int64_t d) { return (n + d - 1) / d; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <class T, int V, int PER>
cudaError_t launch_rows(const NormParams& p, const NormPlan& plan, cudaStream_t stream) {
    norm_kernel<T, V, PER><<<static_cast<unsigned>(plan.chunks), 256, 0, stream>>>(p, plan.group, plan.chunk);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_type(const NormParams& p, const NormPlan& plan, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    if (plan.per == 0) {
        norm_long_kernel<T><<<static_cast<unsigned>(plan.chunks), 256, 0, stream>>>(p);
        return cudaGetLastError();
    }
    if (plan.vec == 1) return plan.per <= 4 ? launch_rows<T, 1, 4>(p, plan, stream) : launch_rows<T, 1, 16>(p, plan, stream);
    switch (plan.per) {
        case 1: return launch_rows<T, V, 1>(p, plan, stream);
        case 2: return launch_rows<T, V, 2>(p, plan, stream);
        case 4: return launch_rows<T, V, 4>(p, plan, stream);
        default: return launch_rows<T, V, 8>(p, plan, stream);
    }
}

template <class T, int V, int PER, int NT>
cudaError_t launch_grad_rows(const GradArgs& a, const NormPlan& plan, cudaStream_t stream) {
    auto* kernel = norm_grad_kernel<T, V, PER, NT>;
    const int smem = NT / std::max(plan.group, 32) * 2 * a.tile * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<dim3(static_cast<unsigned>(plan.chunks), plan.tiles), NT, smem, stream>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_grad_type(const GradArgs& a, const NormPlan& plan, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    if (a.sums) {
        norm_sums_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(a.p.R, int64_t(a.p.sms) * 8)), 256, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (plan.vec == 1) return plan.per <= 4 ? launch_grad_rows<T, 1, 4, 256>(a, plan, stream) : launch_grad_rows<T, 1, 16, 256>(a, plan, stream);
    if (plan.per == 1) return launch_grad_rows<T, V, 1, 256>(a, plan, stream);
    if (plan.per == 2) return launch_grad_rows<T, V, 2, 256>(a, plan, stream);
    return launch_grad_rows<T, V, 4, 256>(a, plan, stream);
}

}  // namespace

NormPlan plan_norm(bool grad, const NormParams& p) {
    NormPlan d{};
    const int size = p.type == PT_F32 ? 4 : 2, v = 16 / size;
    // whole 16-byte loads of every operand
    const bool vec = p.F % v == 0 && p.ldx % v == 0 && aligned16(p.x) && (!p.out || (p.ldo % v == 0 && aligned16(p.out))) &&
                     (!grad || (p.ldy % v == 0 && aligned16(p.dy))) && aligned16(p.weight) && aligned16(p.bias);
    d.vec = vec ? v : 1;
    d.threads = 256;
    const int64_t loads = ceil_to(p.F, d.vec);
    const int most = vec ? (grad ? 4 : 8) : 16;
    d.tiles = 1;
    // a warp's row in registers, or as few threads as hold it; short rows take less than a warp
    d.group = 8;
    const int warp_most = vec ? (grad ? 2 : most) : (loads <= 128 ? 4 : 16);
    while (d.group < 32 && d.group < loads) d.group *= 2;
    while (d.group < 256 && int64_t(d.group) * warp_most < loads) d.group *= 2;
    int64_t per = ceil_to(loads, d.group);
    if (per > most) {
        if (grad) {
            d.tiles = static_cast<int32_t>(ceil_to(per, most));
            per = most;
            d.sums_bytes = ceil_to(p.R * 8, 256) * 256;
        } else {
            per = 0;
        }
    }
    d.per = 1;
    if (!vec) d.per = per <= 4 ? 4 : 16;
    else while (d.per < per) d.per *= 2;
    if (per == 0) d.per = 0;
    const int64_t groups = d.per == 0 ? 1 : d.threads / d.group;
    const int64_t most_blocks = grad ? std::max<int64_t>(int64_t(p.sms) * 4 / d.tiles, 1) : int64_t(p.sms) * 8;
    d.chunk = std::max<int64_t>(ceil_to(ceil_to(p.R, most_blocks), groups) * groups, groups);
    d.chunks = ceil_to(p.R, d.chunk);
    if (d.per == 0) d.chunks = std::min<int64_t>(p.R, most_blocks);
    if (grad) d.partial_bytes = ceil_to(d.chunks * 4 * p.F * 4, 256) * 256;
    return d;
}

cudaError_t launch_norm(const NormParams& p, const NormPlan& plan, cudaStream_t stream) {
    if (p.type == PT_F32) return launch_type<float>(p, plan, stream);
    if (p.type == PT_F16) return launch_type<__half>(p, plan, stream);
    return launch_type<__nv_bfloat16>(p, plan, stream);
}

cudaError_t launch_norm_grad(const NormParams& p, const NormPlan& plan, cudaStream_t stream) {
    GradArgs a{};
    a.p = p;
    a.group = plan.group;
    a.tile = static_cast<int32_t>(std::min<int64_t>(p.F, int64_t(plan.group) * plan.per * plan.vec));
    a.chunk = plan.chunk;
    a.sums = plan.sums_bytes > 0 ? reinterpret_cast<float*>(p.ws) : nullptr;
    a.partials = reinterpret_cast<float*>(p.ws + plan.sums_bytes);
    cudaError_t e;
    if (p.type == PT_F32) e = launch_grad_type<float>(a, plan, stream);
    else if (p.type == PT_F16) e = launch_grad_type<__half>(a, plan, stream);
    else e = launch_grad_type<__nv_bfloat16>(a, plan, stream);
    if (e != cudaSuccess || plan.chunks < 2 || (!p.dweight && !p.dbias)) return e;
    const bool by_start = p.S >= plan.chunks;
    const dim3 grid(static_cast<unsigned>(by_start ? plan.chunks - 1 : p.S), static_cast<unsigned>(std::min<int64_t>(ceil_to(2 * p.F, 32), 16384)));
    norm_add_kernel<<<grid, 256, 0, stream>>>(a, by_start);
    return cudaGetLastError();
}

}  // namespace segred

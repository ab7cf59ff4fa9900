// seg_norm.cu -- layer norm of the rows of segments (see seg_norm.cuh).
//
// A group of threads has a row, in registers: one read of it serves the mean,
// then the centred squares (no difference of large sums), then the result;
// a mean that is large beside the spread is corrected in between (see is_far).
// Groups of up to 32 threads add with shuffles, larger ones through shared
// memory and a barrier of their own.  Everything is float32 and rounded once.
//
// What bounds it: memory, once a row costs few instructions and its loads are on
// their way while others are added up.  16 values of a row per thread, its
// weights in registers over a run of rows of one segment, two values an
// instruction, and a ring of rows in shared memory that every thread fills and
// reads for itself.  32,768 x 2,048 bfloat16, float32 weights: forward 42 us = 6.4
// TB/s (a warp or two a row, weights from L1 for each row, value by value: 84),
// backward 72 to 74 us = 5.5 TB/s (122), 77 with the kernel that adds the parts.
// 1,000,000 x 64 float32 in 50 segments: 91 us = 5.6 TB/s and 126 us = 6.1 TB/s.
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
#include <type_traits>

#include "seg_common.cuh"
#include "seg_norm.cuh"
#include "seg_product.cuh"
#include "tc.cuh"

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

// Two values that one instruction works on (a value at a time the backward pass
// took 28 instructions a value, 32,768 x 2,048 bfloat16 79 us).
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// 16 bytes of values of a thread.  A: they lie on a border of 16 bytes, and rows
// are whole numbers of them.  Else they are G values apart, neighbours those of
// the neighbouring threads (16-bit values may lie between two words, and a warp's
// neighbouring ones are a request of few sectors), and a row's last ones may be
// there in part; the others count as 0.
template <class T, bool A, int G = 1> struct Pack {
    static constexpr int V = 16 / sizeof(T), H = V / 2;
    static constexpr int NEXT = A ? V : 1, STEP = A ? 1 : G;       // values from a thread's first to the next thread's, to its own next one
    using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
    uint4 raw;
    // n: values from p on that there are in the row
    __device__ __forceinline__ void load(const T* p, int n) {
        if constexpr (A) {
            raw = __ldg(reinterpret_cast<const uint4*>(p));
        } else {
            const Bits* from = reinterpret_cast<const Bits*>(p);
            Bits x[V];
            if (n > (V - 1) * STEP) {
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = __ldg(from + i * STEP);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = i * STEP < n ? __ldg(from + i * STEP) : Bits(0);
            }
            if constexpr (sizeof(T) == 4) raw = make_uint4(x[0], x[1], x[2], x[3]);
            else raw = make_uint4(x[0] | uint32_t(x[1]) << 16, x[2] | uint32_t(x[3]) << 16, x[4] | uint32_t(x[5]) << 16, x[6] | uint32_t(x[7]) << 16);
        }
    }
    __device__ __forceinline__ void store(T* p, int n) const {
        if constexpr (A) {
            *reinterpret_cast<uint4*>(p) = raw;
        } else {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            Bits* to = reinterpret_cast<Bits*>(p);
            auto value = [&](int i) { return sizeof(T) == 4 ? static_cast<Bits>(w[i & 3]) : static_cast<Bits>(w[i / 2] >> (i % 2 * 16)); };
            if (n > (V - 1) * STEP) {
#pragma unroll
                for (int i = 0; i < V; ++i) to[i * STEP] = value(i);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i * STEP < n) to[i * STEP] = value(i);
            }
        }
    }
    __device__ __forceinline__ void widen(float2 (&f)[H]) const {
        if constexpr (sizeof(T) == 4) {
            f[0] = make_float2(__uint_as_float(raw.x), __uint_as_float(raw.y));
            f[1] = make_float2(__uint_as_float(raw.z), __uint_as_float(raw.w));
        } else {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
                else f[k] = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            }
        }
    }
    __device__ __forceinline__ void narrow(const float2 (&f)[H]) {
        if constexpr (sizeof(T) == 4) {
            raw = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w[k]) : "f"(f[k].x), "f"(f[k].y));
                else asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(w[k]) : "f"(f[k].x), "f"(f[k].y));
            }
            raw = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// The rows of a group's next windows, on their way to shared memory while it works
// on these: a ring of D slots of ROWS rows of PER packs a thread.  (Those of which
// shared memory does not hold two are loaded when they are needed.)
template <int PACKS, int NT> constexpr int ring_slots() {      // fewer bytes of a slot want more of them
    return PACKS == 1 ? 6 : PACKS <= 4 && NT == 256 ? 4 : PACKS == 2 ? 4 : PACKS <= 4 ? 3 : 2;
}
template <class T, bool A, int G, int PER, int ROWS, int NT, int ROW_BYTES>
struct RingBase {
    static constexpr int D = ring_slots<PER * ROWS, NT>(), SLOT = NT / G * ROWS * ROW_BYTES;
    static constexpr bool ASYNC = D * SLOT <= 200 * 1024;
    static constexpr int BYTES = ASYNC ? D * SLOT : 0;
    uint32_t base, at, to;      // the first slot, the one to read and the one to fetch into
    __device__ __forceinline__ explicit RingBase(uint32_t first) : base(first), at(first), to(first) {}
    __device__ __forceinline__ void fetched() {
        asm volatile("cp.async.commit_group;" ::: "memory");
        to = to == base + (D - 1) * SLOT ? base : to + SLOT;
    }
    __device__ __forceinline__ void got() { at = at == base + (D - 1) * SLOT ? base : at + SLOT; }
    __device__ __forceinline__ void landed() const { asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory"); }
};

// Aligned rows: every thread copies and reads nothing but its own packs, so that no
// barrier is needed.
template <class T, bool A, int G, int PER, int ROWS, int NT>
struct Ring : RingBase<T, A, G, PER, ROWS, NT, G * PER * 16> {
    using B = RingBase<T, A, G, PER, ROWS, NT, G * PER * 16>;
    __device__ __forceinline__ explicit Ring(unsigned char* memory) : B(smem_u32(memory) + threadIdx.x * 16) {}
    // row q of the thread's, whose own part of it begins at `from`
    __device__ __forceinline__ void fetch(int q, const T* from, int left, const void*) const {
        if constexpr (B::ASYNC)
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (j * G * Pack<T, A>::V < left)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(this->to + (q * PER + j) * NT * 16), "l"(from + j * G * Pack<T, A>::V) : "memory");
    }
    // the slot to read is there
    __device__ __forceinline__ void wait() const { this->landed(); }
    // pack j of row q, which memory has at `from`
    __device__ __forceinline__ void get(int q, int j, const T* from, uint32_t, int n, float2 (&f)[Pack<T, A>::H]) const {
        Pack<T, A> x;
        if constexpr (B::ASYNC)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.raw.x), "=r"(x.raw.y), "=r"(x.raw.z), "=r"(x.raw.w) : "r"(this->at + (q * PER + j) * NT * 16) : "memory");
        else x.load(from, n);
        x.widen(f);
    }
    // packs that are never fetched read as zeros
    __device__ __forceinline__ void clear(int q, int j) const {
        if constexpr (B::ASYNC)
            for (int d = 0; d < B::D; ++d)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(this->base + d * B::SLOT + (q * PER + j) * NT * 16), "r"(0) : "memory");
    }
};

// Other rows: the aligned 16 bytes that a row lies in are copied, 16 each, and the
// group's threads read the row's values from wherever it begins in them (200,000 x
// 333 float32 forward 97 us, loaded when they are needed 198; bfloat16 93 and 128,
// where each value's own load, mask and store are what bounds it).
template <class T, int G, int PER, int ROWS, int NT>
struct Ring<T, false, G, PER, ROWS, NT> : RingBase<T, false, G, PER, ROWS, NT, (G * PER + 1) * 16> {
    static constexpr int ROW_BYTES = (G * PER + 1) * 16, SIZE = sizeof(T);
    using B = RingBase<T, false, G, PER, ROWS, NT, ROW_BYTES>;
    using P = Pack<T, false, G>;
    __device__ __forceinline__ explicit Ring(unsigned char* memory) : B(smem_u32(memory)) {}
    static __device__ __forceinline__ uint32_t row_at(int q) { return (threadIdx.x / G * ROWS + q) * ROW_BYTES; }
    // first: the tensor's first value.  Nothing before it or behind the row's last one is read.
    __device__ __forceinline__ void fetch(int q, const T* from, int left, const void* first) const {
        if constexpr (B::ASYNC) {
            const int t = threadIdx.x % G;
            const uintptr_t begin = reinterpret_cast<uintptr_t>(from - t), end = begin + min(left + t, G * PER * P::V) * SIZE;
            const uintptr_t unit = (begin & ~uintptr_t(15)) + t * 16;
#pragma unroll
            for (int k = 0; k <= PER; ++k) {
                const uintptr_t u = unit + k * G * 16;
                if (u >= end || (k == PER && t > 0)) break;
                const uint32_t dst = this->to + row_at(q) + t * 16 + k * G * 16;
                if (u >= reinterpret_cast<uintptr_t>(first)) {
                    const int bytes = end - u < 16 ? static_cast<int>(end - u) : 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(u), "r"(bytes) : "memory");
                } else {
                    for (int i = static_cast<int>(begin - u); i < 16 && u + i < end; i += SIZE) {
                        if constexpr (SIZE == 2) asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + i), "h"(__ldg(reinterpret_cast<const uint16_t*>(u + i))) : "memory");
                        else asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + i), "r"(__ldg(reinterpret_cast<const uint32_t*>(u + i))) : "memory");
                    }
                }
            }
        }
    }
    // (nor has a thread of the group anything left to read of the slot before)
    __device__ __forceinline__ void wait() const {
        this->landed();
        if constexpr (G <= 32) __syncwarp();
        else if constexpr (G == NT) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + int(threadIdx.x) / G), "n"(G) : "memory");
    }
    // low: the last bits of the address of the row's first value
    __device__ __forceinline__ void get(int q, int j, const T* from, uint32_t low, int n, float2 (&f)[P::H]) const {
        if constexpr (B::ASYNC) {
            const uint32_t src = this->at + row_at(q) + (low & 15) + (threadIdx.x % G) * SIZE + j * G * 16;
            float x[P::V];
#pragma unroll
            for (int i = 0; i < P::V; ++i) {
                x[i] = 0.0f;
                if (i * G < n) x[i] = value(src + i * G * SIZE);
            }
#pragma unroll
            for (int k = 0; k < P::H; ++k) f[k] = make_float2(x[2 * k], x[2 * k + 1]);
        } else {
            P x;
            x.load(from, n);
            x.widen(f);
        }
    }
    static __device__ __forceinline__ float value(uint32_t src) {
        if constexpr (SIZE == 4) {
            float v;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(src) : "memory");
            return v;
        } else {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src) : "memory");
            if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(uint32_t(v) << 16);
            else return __half2float(__ushort_as_half(v));
        }
    }
    __device__ __forceinline__ void clear(int, int) const {}
};

// A pack of values of weight_type at element `at`, n of them from there on in the row.
template <class T, bool A, int G = 1>
__device__ __forceinline__ void load_weights(const void* w, bool wide, int64_t at, int n, float2 (&f)[Pack<T, A>::H]) {
    if (!wide) {
        Pack<T, A, G> x;
        x.load(static_cast<const T*>(w) + at, n);
        x.widen(f);
        return;
    }
    const float* p = static_cast<const float*>(w) + at;
#pragma unroll
    for (int i = 0; i < Pack<T, A>::H; i += 2) {
        Pack<float, A, G> x;
        float2 y[2];
        x.load(p + 2 * i * Pack<T, A, G>::STEP, n - 2 * i * Pack<T, A, G>::STEP);
        x.widen(y);
        f[i] = y[0], f[i + 1] = y[1];
    }
}
template <class T, bool A, int G = 1>
__device__ __forceinline__ void store_weights(void* out, bool wide, int64_t at, int n, const float2 (&f)[Pack<T, A>::H]) {
    if (!wide) {
        Pack<T, A, G> x;
        x.narrow(f);
        x.store(static_cast<T*>(out) + at, n);
        return;
    }
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int i = 0; i < Pack<T, A>::H; i += 2) {
        Pack<float, A, G> x;
        const float2 y[2] = {f[i], f[i + 1]};
        x.narrow(y);
        x.store(p + 2 * i * Pack<T, A, G>::STEP, n - 2 * i * Pack<T, A, G>::STEP);
    }
}
template <class T>
__device__ __forceinline__ float load_weight(const void* w, bool wide, int64_t at) {
    return wide ? __ldg(static_cast<const float*>(w) + at) : to_float<T>(static_cast<const T*>(w)[at]);
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
// before: the segment of an earlier row, or -1.  It is mostly the next one: two
// loads at once where the search is a chain of them.
__device__ __forceinline__ Run run_of(const NormParams& p, int64_t r, int64_t before = -1) {
    if (!p.offsets) return {0, 0, p.R};
    if (before >= 0 && before + 2 <= p.S) {
        const int64_t begin = offset_at(p, before + 1), end = offset_at(p, before + 2);
        if (begin <= r && r < end) return {before + 1, begin, end};
    }
    int64_t lo = -1, hi = p.S + 1;      // the last offset at or before r; the first one after it
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

// Sums of N values over the G threads of a row, to all of them: within a warp
// with shuffles, then over the row's warps through shared memory, at a barrier of
// theirs.  `red`: [2][warps of the block][N], used in turns.
template <int G, int NT, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
    for (int d = (G < 32 ? G : 32) / 2; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    if constexpr (G > 32) {
        constexpr int WARPS = G / 32;
        const int warp = threadIdx.x >> 5;
        float* at = red + turn * (NT / 32) * N;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) at[warp * N + i] = v[i];
        if constexpr (G == NT) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WARPS), "n"(G) : "memory");
        at += warp / WARPS * WARPS * N;
        if constexpr (WARPS >= 16) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = at[(threadIdx.x % WARPS) * N + i];
#pragma unroll
            for (int d = WARPS / 2; d > 0; d >>= 1)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += at[w * N + i];
        }
        turn ^= 1;
    }
}

// A row's first mean is off by its sum's roundings and 1 / F's: by some units of
// 2^-24 of the values' mean size, which is at most the standard deviation and
// |mean|.  Where |mean| is at most half the deviation z is off by as little.  Else
// rstd would enlarge it, by up to 1 / sqrt(eps) = 316 (41 equal values 1,000: z =
// 0.02, not 0), and the mean is corrected: what it leaves of the values, d = x -
// mean, is exact where they are near one another, and small, so
//   shift = sum d / F,  variance = (sum d^2 - shift sum d) / F
// lose nothing; of equal values the shift is d itself and the variance 0.  (Asked
// for each row: 8,192 x 5,000 bfloat16 40.5 -> 43 us, 200,000 x 333 89 -> 93, 1,000,000
// x 64 47 -> 46.5; where all rows are far 53, 97 and 51; a sum more in every row,
// near or far, 48.5, 96 and 54.)
// var: the variance about the first mean, with eps.
__device__ __forceinline__ bool is_far(float mean, float var) { return 4.0f * mean * mean > var; }
// From the sum of d and that of d^2, which becomes the corrected one.  inv is 1 /
// F rounded; the quotient's remainder by one fma corrects it to the last bit
// (Markstein, 1990), which equal values need.
__device__ __forceinline__ float shift_of(float sum, float& squares, float columns, float inv) {
    const float q = sum * inv, shift = fmaf(fmaf(-q, columns, sum), inv, q), left = fmaf(-shift, sum, squares);
    squares = left < 0.0f ? 0.0f : left;       // (NaN stays NaN)
    return shift;
}

// Blocks of an SM, by the values that a thread holds of rows and weights.
constexpr int resident(int threads, int values) { return threads > 256 ? 1 : values > 48 ? 2 : values > 24 ? 3 : 4; }
// Values of a row that a thread has, and rows at a time: the forward pass takes
// two, whose sums' chains overlap, of 16 values each; one of 32; and one of 16-bit
// values that are not aligned, with three blocks an SM for two (200,000 x 333
// bfloat16 92 -> 86 us; float32 97 -> 93, but 50,000 x 1,001 68 -> 73).  The backward
// pass has sums to keep as well: two where a thread has one pack of a row
// (1,000,000 rows of 64 bfloat16 columns 91.7 -> 81.7 us, of 32 83.6 -> 69.3), else one.
constexpr int ROW_VALUES = 16;
constexpr int forward_rows(bool aligned, int size, int threads, int per) {
    return per * (16 / size) > ROW_VALUES || (!aligned && size == 2 && threads == 256) ? 1 : 2;
}
constexpr int grad_rows(int per) { return per == 1 ? 2 : 1; }

// G threads a row, U rows of a group at a time.
template <class T, bool A, int G, int PER, int U, int NT>
__global__ void __launch_bounds__(NT, resident(NT, Pack<T, A>::V * PER * (U + 2))) norm_kernel(const __grid_constant__ NormParams p, int64_t chunk) {
    using R = Ring<T, A, G, PER, U, NT>;
    using P = Pack<T, A, G>;
    constexpr int V = P::V, GROUPS = NT / G, STEP = G * V, H = V / 2;
    static_assert(NT <= 512 && R::ASYNC, "a run's weights stay in registers, the next rows are on their way to shared memory");
    __shared__ float red[2 * NT / 32 * U];
    extern __shared__ __align__(16) unsigned char ring_memory[];
    R ring(ring_memory);
    const int t = threadIdx.x % G, g = threadIdx.x / G;
    const int64_t c0 = blockIdx.x * chunk;
    const int n = static_cast<int>(min(chunk, p.R - c0));                 // rows of the chunk
    const int left = static_cast<int>(p.F) - t * P::NEXT;                 // pack j is in the row where j STEP < left
    const float inv = 1.0f / static_cast<float>(p.F);
    const bool wide = p.weight_type == PT_F32;
    const int64_t next = GROUPS * p.ldx;                                  // from a group's row to its next one
    const T* pf = static_cast<const T*>(p.x) + (c0 + g) * p.ldx + t * P::NEXT;
    uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(pf - t * P::NEXT));
    const uint32_t low_next = static_cast<uint32_t>(next * sizeof(T));
    auto fetch = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u * GROUPS < n) ring.fetch(u, pf, left, p.x);
            pf += next;
        }
        ring.fetched();
    };
    for (int d = 0; d < R::D - 1; ++d) fetch(d * GROUPS * U + g);
    int turn = 0, run_end = 0;      // of the chunk's rows
    int64_t at = 0, segment = -1;
    bool used = false;
    float2 kept_w[PER][H], kept_b[PER][H];
    auto read_weights = [&](int j, float2 (&w)[H], float2 (&b)[H]) {
#pragma unroll
        for (int k = 0; k < H; ++k) w[k] = pair(1.0f), b[k] = pair(0.0f);
        if (p.weight) load_weights<T, A, G>(p.weight, wide, at + j * STEP, left - j * STEP, w);
        if (p.bias) load_weights<T, A, G>(p.bias, wide, at + j * STEP, left - j * STEP, b);
    };
    auto find_run = [&](int i) {
        const Run run = run_of(p, c0 + i, segment);
        segment = run.s;
        run_end = static_cast<int>(min(run.end - c0, int64_t(n)));
        used = run.s >= 0;
        at = run.s * p.F + t * P::NEXT;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (used && j * STEP < left) read_weights(j, kept_w[j], kept_b[j]);
    };
    if (g < n) find_run(g);        // while the first rows are on their way
    for (int base = 0; base < n; base += GROUPS * U) {
        float2 f[U][PER][H];
        float sum[U], sq[U];
        ring.wait();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = base + u * GROUPS + g < n;
            float2 all = pair(0.0f);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (in && j * STEP < left) {
                    ring.get(u, j, nullptr, low + u * low_next, left - j * STEP, f[u][j]);
#pragma unroll
                    for (int i = 0; i < H; ++i) all = __fadd2_rn(all, f[u][j][i]);
                } else {
#pragma unroll
                    for (int i = 0; i < H; ++i) f[u][j][i] = pair(0.0f);
                }
            }
            sum[u] = all.x + all.y;
        }
        ring.got();
        low += U * low_next;
        fetch(base + (R::D - 1) * GROUPS * U + g);
        group_sum<G, NT, U>(sum, red, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] *= inv;
            float2 all = pair(0.0f);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (j * STEP >= left) continue;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    f[u][j][i] = __fadd2_rn(f[u][j][i], pair(-sum[u]));
                    if constexpr (!A) {
                        if (2 * i * P::STEP >= left - j * STEP) f[u][j][i].x = 0.0f;
                        if ((2 * i + 1) * P::STEP >= left - j * STEP) f[u][j][i].y = 0.0f;
                    }
                    all = __ffma2_rn(f[u][j][i], f[u][j][i], all);
                }
            }
            sq[u] = all.x + all.y;
        }
        group_sum<G, NT, U>(sq, red, turn);
        float var[U];                   // and eps
        bool far[U], any = false;       // the same in all threads of a row
#pragma unroll
        for (int u = 0; u < U; ++u) {
            var[u] = fmaf(sq[u], inv, p.eps);
            any |= far[u] = is_far(sum[u], var[u]);
        }
        if constexpr (G < 32) any = __any_sync(0xffffffffu, any);
        if (__builtin_expect(any, 0)) {
            float rest[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 all = pair(0.0f);
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j * STEP < left)
#pragma unroll
                        for (int i = 0; i < H; ++i) all = __fadd2_rn(all, f[u][j][i]);
                rest[u] = all.x + all.y;
            }
            group_sum<G, NT, U>(rest, red, turn);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!far[u]) continue;
                const float shift = shift_of(rest[u], sq[u], static_cast<float>(p.F), inv);
                sum[u] += shift;
                var[u] = fmaf(sq[u], inv, p.eps);
#pragma unroll
                for (int j = 0; j < PER; ++j)
#pragma unroll
                    for (int i = 0; i < H; ++i) f[u][j][i] = __fadd2_rn(f[u][j][i], pair(-shift));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * GROUPS + g;
            if (i >= n) break;
            const int64_t r = c0 + i;
            if (i >= run_end) find_run(i);
            const float rstd = rsqrtf(var[u]);
            if (t == 0) {
                if (p.mean) p.mean[r] = used ? sum[u] : 0.0f;
                if (p.rstd) p.rstd[r] = used ? rstd : 0.0f;
            }
            T* y = static_cast<T*>(p.out) + r * p.ldo + t * P::NEXT;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (j * STEP >= left) continue;
#pragma unroll
                for (int k = 0; k < H; ++k) f[u][j][k] = used ? __ffma2_rn(__fmul2_rn(f[u][j][k], pair(rstd)), kept_w[j][k], kept_b[j][k]) : pair(0.0f);
                P o;
                o.narrow(f[u][j]);
                o.store(y + j * STEP, left - j * STEP);
            }
        }
    }
}

// Sum of one value over the block (256 threads), to all of them.
__device__ __forceinline__ float block_sum(float v, float* red) {
    float x[1] = {v};
    int turn = 0;
    __syncthreads();
    group_sum<256, 256, 1>(x, red, turn);
    return x[0];
}

// Wide rows: a block's row stays in the ring of shared memory and is read from
// there for each pass over it, so that few registers and two blocks of an SM are
// enough to have one row on its way while others are added up.  What bounds it are
// the weights, which come from L2 for each row (2,000 x 20,000 bfloat16 with
// float32 weights 54 us; 5,000 x 9,000, which go by registers, 58 so and 43).
constexpr int WIDE_THREADS = 512, WIDE_SLOTS = 3;
template <class T>
__global__ void __launch_bounds__(WIDE_THREADS, 2) norm_wide_kernel(const __grid_constant__ NormParams p, int64_t chunk) {
    constexpr int V = Pack<T, true>::V, H = V / 2, NT = WIDE_THREADS;
    __shared__ float red[2 * NT / 32];
    extern __shared__ __align__(16) unsigned char ring_memory[];
    const int t = threadIdx.x, packs = static_cast<int>(p.F / V);
    const int64_t c0 = blockIdx.x * chunk;
    const int n = static_cast<int>(min(chunk, p.R - c0));
    const float inv = 1.0f / static_cast<float>(p.F);
    const bool wide = p.weight_type == PT_F32;
    const uint32_t base = smem_u32(ring_memory) + t * 16, slot_bytes = packs * 16;
    const T* px = static_cast<const T*>(p.x) + c0 * p.ldx;
    auto fetch = [&](int i) {
        if (i < n)
            for (int j = t; j < packs; j += NT)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + i % WIDE_SLOTS * slot_bytes + (j - t) * 16), "l"(px + i * p.ldx + j * V) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int d = 0; d < WIDE_SLOTS - 1; ++d) fetch(d);
    int turn = 0;
    Run run;
    for (int i = 0; i < n; ++i) {
        fetch(i + WIDE_SLOTS - 1);        // (a slot that this thread was through with a row ago)
        asm volatile("cp.async.wait_group %0;" ::"n"(WIDE_SLOTS - 1) : "memory");
        const uint32_t slot = base + i % WIDE_SLOTS * slot_bytes;
        auto get = [&](int j, float2 (&f)[H]) {
            Pack<T, true> x;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.raw.x), "=r"(x.raw.y), "=r"(x.raw.z), "=r"(x.raw.w) : "r"(slot + (j - t) * 16) : "memory");
            x.widen(f);
        };
        float2 f[H], all = pair(0.0f);
        for (int j = t; j < packs; j += NT) {
            get(j, f);
#pragma unroll
            for (int k = 0; k < H; ++k) all = __fadd2_rn(all, f[k]);
        }
        float sum[1] = {all.x + all.y};
        group_sum<NT, NT, 1>(sum, red, turn);
        const float mean = sum[0] * inv;
        all = pair(0.0f);
        for (int j = t; j < packs; j += NT) {
            get(j, f);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                f[k] = __fadd2_rn(f[k], pair(-mean));
                all = __ffma2_rn(f[k], f[k], all);
            }
        }
        sum[0] = all.x + all.y;
        group_sum<NT, NT, 1>(sum, red, turn);
        float shift = 0.0f;
        if (is_far(mean, fmaf(sum[0], inv, p.eps))) {
            all = pair(0.0f);
            for (int j = t; j < packs; j += NT) {
                get(j, f);
#pragma unroll
                for (int k = 0; k < H; ++k) all = __fadd2_rn(all, __fadd2_rn(f[k], pair(-mean)));
            }
            float rest[1] = {all.x + all.y};
            group_sum<NT, NT, 1>(rest, red, turn);
            shift = shift_of(rest[0], sum[0], static_cast<float>(p.F), inv);
        }
        const float rstd = rsqrtf(fmaf(sum[0], inv, p.eps));
        const int64_t r = c0 + i;
        if (r >= run.end) run = run_of(p, r, run.s);
        const bool used = run.s >= 0;
        if (t == 0) {
            if (p.mean) p.mean[r] = used ? mean + shift : 0.0f;
            if (p.rstd) p.rstd[r] = used ? rstd : 0.0f;
        }
        T* y = static_cast<T*>(p.out) + r * p.ldo;
        for (int j = t; j < packs; j += NT) {
            float2 w[H], b[H];
#pragma unroll
            for (int k = 0; k < H; ++k) w[k] = pair(1.0f), b[k] = pair(0.0f);
            if (used && p.weight) load_weights<T, true>(p.weight, wide, run.s * p.F + j * V, V, w);
            if (used && p.bias) load_weights<T, true>(p.bias, wide, run.s * p.F + j * V, V, b);
            get(j, f);
#pragma unroll
            for (int k = 0; k < H; ++k) f[k] = used ? __ffma2_rn(__fmul2_rn(__fadd2_rn(__fadd2_rn(f[k], pair(-mean)), pair(-shift)), pair(rstd)), w[k], b[k]) : pair(0.0f);
            Pack<T, true> o;
            o.narrow(f);
            o.store(y + j * V, V);
        }
    }
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
        if (r >= run.end) run = run_of(p, r, run.s);
        float sum = 0.0f, rest = 0.0f, sq = 0.0f;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) sum += to_float<T>(x[c]);
        const float mean = block_sum(sum, red) * inv;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) {
            const float d = to_float<T>(x[c]) - mean;
            rest += d;
            sq = fmaf(d, d, sq);
        }
        rest = block_sum(rest, red);
        sq = block_sum(sq, red);
        // (the reads bound this kernel: every row's mean is corrected)
        const float shift = shift_of(rest, sq, static_cast<float>(p.F), inv);
        const float rstd = rsqrtf(fmaf(sq, inv, p.eps));
        const bool used = run.s >= 0;
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = used ? mean + shift : 0.0f;
            if (p.rstd) p.rstd[r] = used ? rstd : 0.0f;
        }
        T* y = static_cast<T*>(p.out) + r * p.ldo;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) {
            const float w = used && p.weight ? load_weight<T>(p.weight, wide, run.s * p.F + c) : 1.0f;
            const float b = used && p.bias ? load_weight<T>(p.bias, wide, run.s * p.F + c) : 0.0f;
            y[c] = from_float<T>(used ? fmaf((to_float<T>(x[c]) - mean - shift) * rstd, w, b) : 0.0f);
        }
    }
}

// ---------------------------------------------------------------------------

struct GradArgs {
    NormParams p;
    int32_t tile;               // columns of a tile
    int32_t clear;              // segments without rows are cleared at a block's end
    int64_t chunk;
    float* sums;                // [R][2]: sum(g), sum(g z) of each row, or NULL: a block has all columns, or dx is not wanted
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
        if (r >= run.end) run = run_of(p, r, run.s);
        if (run.s < 0) continue;
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        const T* dy = static_cast<const T*>(p.dy) + r * p.ldy;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < p.F; c += 256) {
            const float gr = to_float<T>(dy[c]) * (p.weight ? load_weight<T>(p.weight, wide, run.s * p.F + c) : 1.0f);
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

// Which of the segments s, one of each lane of a warp, are below `end` and have no rows.
__device__ __forceinline__ uint32_t without_rows(const NormParams& p, int64_t s, int64_t end) {
    return __ballot_sync(0xffffffffu, s < end && offset_at(p, min(s, p.S)) >= offset_at(p, min(s + 1, p.S)));
}

// The sums of segments without rows, columns c0 to c1: a warp looks at 32 segments
// at once.  (At a block's end: before its rows this cost them registers, 5,000 x
// 9,001 float32 187 -> 304 us.)
__device__ __forceinline__ void clear_empty(const NormParams& p, int c0, int c1) {
    const int64_t each = (p.S + gridDim.x - 1) / gridDim.x, s1 = min((blockIdx.x + 1) * each, p.S);
    const int lane = threadIdx.x & 31;
    for (int64_t s0 = blockIdx.x * each + (threadIdx.x & ~31); s0 < s1; s0 += blockDim.x) {
        const int64_t s = s0 + lane;
        for (uint32_t none = without_rows(p, s, s1); none; none &= none - 1) {
            const int64_t at = (s0 + __ffs(none) - 1) * p.F;
            for (int c = c0 + lane; c < c1; c += 32) {
                if (p.dweight) store_weight(p.dweight, p.weight_type, at + c, 0.0f);
                if (p.dbias) store_weight(p.dbias, p.weight_type, at + c, 0.0f);
            }
        }
    }
}

// The same where the blocks that the rows need are few for the sums that may have
// to be cleared (see plan_norm): a warp takes 32 segments and CLEAR_COLUMNS
// columns at a time, 16 bytes a lane where the sums are whole units of those.
// Segments next to one another with all their columns are one piece.
constexpr int CLEAR_COLUMNS = 512;
__global__ void __launch_bounds__(256) norm_clear_kernel(const __grid_constant__ NormParams p, int size, int whole) {
    const int lane = threadIdx.x & 31;
    const int64_t across = (p.F + CLEAR_COLUMNS - 1) / CLEAR_COLUMNS, tiles = (p.S + 31) / 32 * across;
    for (int64_t i = blockIdx.x * int64_t(8) + threadIdx.x / 32; i < tiles; i += gridDim.x * int64_t(8)) {
        const int64_t s0 = i / across * 32, c0 = i % across * CLEAR_COLUMNS, c1 = min(c0 + CLEAR_COLUMNS, p.F);
        uint32_t none = without_rows(p, s0 + lane, p.S);
        while (none) {
            const int at = __ffs(none) - 1, others = across > 1 ? 0 : __ffs(~(none >> at)) - 2;     // segments after the first one
            const int n = others == -2 ? 32 - at : others + 1;
            none &= n == 32 ? 0 : ~(((1u << n) - 1) << at);
            const int64_t begin = ((s0 + at) * p.F + c0) * size, end = ((s0 + at + n - 1) * p.F + c1) * size;
            for (void* sums : {p.dweight, p.dbias}) {
                if (!sums) continue;
                char* to = static_cast<char*>(sums);
                if (whole)
                    for (int64_t b = begin + lane * 16; b < end; b += 512) *reinterpret_cast<uint4*>(to + b) = make_uint4(0, 0, 0, 0);
                else if (size == 4)
                    for (int64_t b = begin + lane * 4; b < end; b += 128) *reinterpret_cast<float*>(to + b) = 0.0f;
                else
                    for (int64_t b = begin + lane * 2; b < end; b += 64) *reinterpret_cast<uint16_t*>(to + b) = 0;
            }
        }
    }
}

// A block's windows of U rows of each group follow one another whatever
// segments they are in; a window in which a run ends is worked on once for each
// run that has a row in it.
template <class T, bool A, int G, int PER, int U, int NT>
__global__ void __launch_bounds__(NT, resident(NT, Pack<T, A>::V * PER * (2 * U + 3))) norm_grad_kernel(const __grid_constant__ GradArgs a) {
    using R = Ring<T, A, G, PER, 2 * U, NT>;
    using P = Pack<T, A, G>;
    constexpr int V = P::V, GROUPS = NT / G, STEP = G * V, WINDOW = GROUPS * U, H = V / 2;
    constexpr bool KEEP = NT <= 512 && PER * V <= ROW_VALUES;      // a run's weights stay in registers; a large block has none to spare and reads them again
    __shared__ float red[2 * NT / 32 * 2 * U];
    extern __shared__ __align__(16) unsigned char ring_memory[];
    float* const shared_sums = reinterpret_cast<float*>(ring_memory + R::BYTES);      // [groups of at least a warp][2][tile]
    R ring(ring_memory);
    grid_trigger();
    const NormParams& p = a.p;
    const int t = threadIdx.x % G, g = threadIdx.x / G;
    const int64_t c0 = blockIdx.x * a.chunk;
    const int n = static_cast<int>(min(a.chunk, p.R - c0));
    const int col0 = static_cast<int>(blockIdx.y) * a.tile, F = static_cast<int>(p.F), left = F - col0 - t * P::NEXT;
    const float inv = 1.0f / static_cast<float>(p.F);
    const bool wide = p.weight_type == PT_F32, want_dx = p.out != nullptr, want_dw = p.dweight || p.dbias;
    const int64_t nextx = GROUPS * p.ldx, nexty = GROUPS * p.ldy;
    const T* px = static_cast<const T*>(p.x) + (c0 + g) * p.ldx + col0 + t * P::NEXT;
    const T* pd = static_cast<const T*>(p.dy) + (c0 + g) * p.ldy + col0 + t * P::NEXT;
    auto low_bits = [](const T* row) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)); };
    uint32_t lowx = low_bits(px - t * P::NEXT), lowy = low_bits(pd - t * P::NEXT);
    const uint32_t lowx_next = static_cast<uint32_t>(nextx * sizeof(T)), lowy_next = static_cast<uint32_t>(nexty * sizeof(T));
    auto fetch = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u * GROUPS < n) ring.fetch(2 * u, px, left, p.x), ring.fetch(2 * u + 1, pd, left, p.dy);
            px += nextx;
            pd += nexty;
        }
        ring.fetched();
    };
    if (R::ASYNC) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (j * STEP >= left)
                for (int u = 0; u < U; ++u) ring.clear(2 * u, j), ring.clear(2 * u + 1, j);
        for (int d = 0; d < R::D - 1; ++d) fetch(d * WINDOW + g);
    }
    Run run = run_of(p, c0);
    float2 kept[KEEP ? PER : 1][H], dw[PER][H], db[PER][H];
    auto read_weights = [&](int j, float2 (&w)[H]) {
        if (p.weight && run.s >= 0 && j * STEP < left) {
            load_weights<T, A, G>(p.weight, wide, run.s * p.F + col0 + t * P::NEXT + j * STEP, left - j * STEP, w);
        } else {
#pragma unroll
            for (int i = 0; i < H; ++i) w[i] = pair(1.0f);
        }
    };
    auto weights_of = [&](int j, float2 (&w)[H]) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < H; ++i) w[i] = kept[j][i];
        } else {
            read_weights(j, w);
        }
    };
    int run_end = 0;                   // of the chunk's rows; past its last one where the run goes on
    auto begin = [&] {
        run_end = static_cast<int>(min(run.end - c0, int64_t(n) + 1));
#pragma unroll
        for (int j = 0; j < PER; ++j) {
#pragma unroll
            for (int i = 0; i < H; ++i) dw[j][i] = db[j][i] = pair(0.0f);
            if constexpr (KEEP) read_weights(j, kept[j]);
        }
    };
    begin();
    float next_mean[U], next_rstd[U];
    const float* pm = p.mean + c0 + g;
    const float* pr = p.rstd + c0 + g;
    auto fetch_stats = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next_mean[u] = next_rstd[u] = 0.0f;
            if (i + u * GROUPS < n) next_mean[u] = __ldg(pm + u * GROUPS), next_rstd[u] = __ldg(pr + u * GROUPS);
        }
        pm += WINDOW;
        pr += WINDOW;
    };
    fetch_stats(g);
    const int64_t nexto = GROUPS * p.ldo;
    T* po = static_cast<T*>(p.out) + (c0 + g) * p.ldo + col0 + t * P::NEXT;
    int turn = 0;
    for (int base = 0; base < n; base += WINDOW) {
        const int end = min(base + WINDOW, n);
        float2 kept_z[KEEP ? U : 1][KEEP ? PER : 1][H], kept_dy[KEEP ? U : 1][KEEP ? PER : 1][H];
        float mean[U], rstd[U];
        if (R::ASYNC) ring.wait();
        auto read_values = [&](int u, int j, float2 (&z)[H], float2 (&dy)[H]) {
            ring.get(2 * u, j, px + u * nextx + j * STEP, lowx + u * lowx_next, left - j * STEP, z);
            ring.get(2 * u + 1, j, pd + u * nexty + j * STEP, lowy + u * lowy_next, left - j * STEP, dy);
#pragma unroll
            for (int i = 0; i < H; ++i) z[i] = __fmul2_rn(__fadd2_rn(z[i], pair(-mean[u])), pair(rstd[u]));
        };
        auto values_of = [&](int u, int j, float2 (&z)[H], float2 (&dy)[H]) {
            if constexpr (KEEP) {
#pragma unroll
                for (int i = 0; i < H; ++i) z[i] = kept_z[u][j][i], dy[i] = kept_dy[u][j][i];
            } else {
                read_values(u, j, z, dy);
            }
        };
        auto values_read = [&] {
            if (R::ASYNC) {
                ring.got();
                lowx += U * lowx_next;
                lowy += U * lowy_next;
                fetch(base + (R::D - 1) * WINDOW + g);
            } else {
                px += U * nextx;
                pd += U * nexty;
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[u] = next_mean[u];
            rstd[u] = next_rstd[u];
            if constexpr (KEEP)
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (R::ASYNC || (base + u * GROUPS + g < n && j * STEP < left)) read_values(u, j, kept_z[u][j], kept_dy[u][j]);
        }
        if constexpr (KEEP) values_read();
        fetch_stats(base + WINDOW + g);
        int from = base;               // the window's rows before are done
        for (;;) {
            const int to = min(run_end, end);
            auto in = [&](int u) { return base + u * GROUPS + g >= from && base + u * GROUPS + g < to; };
            // one run's rows of the window; ALL: they are all there (columns that
            // the row does not have count as zeros)
            auto work = [&](auto all) {
                constexpr bool ALL = decltype(all)::value;
                float s[2 * U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float2 s1 = pair(0.0f), s2 = pair(0.0f);
                    if (ALL || in(u))
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            if (!R::ASYNC && j * STEP >= left) continue;
                            float2 w[H], z[H], dy[H];
                            weights_of(j, w);
                            values_of(u, j, z, dy);
#pragma unroll
                            for (int i = 0; i < H; ++i) {
                                const float2 gr = __fmul2_rn(dy[i], w[i]);
                                db[j][i] = __fadd2_rn(db[j][i], dy[i]);
                                dw[j][i] = __ffma2_rn(dy[i], z[i], dw[j][i]);
                                s1 = __fadd2_rn(s1, gr);
                                s2 = __ffma2_rn(gr, z[i], s2);
                            }
                        }
                    s[2 * u] = s1.x + s1.y;
                    s[2 * u + 1] = s2.x + s2.y;
                }
                if (!want_dx) return;
                if (!a.sums) group_sum<G, NT, 2 * U>(s, red, turn);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (!ALL && !in(u)) continue;
                    if (a.sums) {
                        const int64_t r = c0 + base + u * GROUPS + g;
                        s[2 * u] = __ldg(a.sums + 2 * r), s[2 * u + 1] = __ldg(a.sums + 2 * r + 1);
                    }
                    const float2 m1 = pair(-s[2 * u] * inv), m2 = pair(-s[2 * u + 1] * inv), scale = pair(rstd[u]);
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        if (!R::ASYNC && j * STEP >= left) continue;
                        P o;
                        float2 w[H], z[H], dy[H], d[H];
                        weights_of(j, w);
                        values_of(u, j, z, dy);
#pragma unroll
                        for (int i = 0; i < H; ++i) d[i] = __fmul2_rn(scale, __ffma2_rn(z[i], m2, __ffma2_rn(dy[i], w[i], m1)));
                        o.narrow(d);
                        if (j * STEP < left) o.store(po + u * nexto + j * STEP, left - j * STEP);
                    }
                }
            };
            if (run.s >= 0) {
                if (from == base && to == base + WINDOW) work(std::true_type());
                else work(std::false_type());
            } else if (want_dx) {
                // rows in no segment
                const float2 none[H] = {};
                P zero;
                zero.narrow(none);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (in(u) && j * STEP < left) zero.store(po + u * nexto + j * STEP, left - j * STEP);
            }
            if (run_end > end && end < n) break;       // the run goes on in the next window
            if (want_dw && run.s >= 0) {
                // the run's end in this chunk: the groups' sums, of a warp's groups
                // first, then of the warps, each in their order
#pragma unroll
                for (int d = 16; d >= G; d >>= 1) {
#pragma unroll
                    for (int j = 0; j < PER; ++j)
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            for (float* v : {&dw[j][i].x, &dw[j][i].y, &db[j][i].x, &db[j][i].y}) *v += __shfl_xor_sync(0xffffffffu, *v, d);
                }
                const bool whole = run.begin >= c0 && run.end <= c0 + n;
                float* slot_sums = a.partials + (2 * int64_t(blockIdx.x) + (run.begin >= c0 ? 1 : 0)) * 2 * p.F;
                auto put = [&](int which, int c, float v) {
                    void* out = which ? p.dbias : p.dweight;
                    if (!out) return;
                    if (!whole) slot_sums[which * p.F + c] = v;
                    else store_weight(out, p.weight_type, run.s * p.F + c, v);
                };
                if constexpr (G == NT) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int c = col0 + t * P::NEXT + j * STEP;
                        if (j * STEP >= left) continue;
                        if (whole) {
                            if (p.dweight) store_weights<T, A, G>(p.dweight, wide, run.s * p.F + c, left - j * STEP, dw[j]);
                            if (p.dbias) store_weights<T, A, G>(p.dbias, wide, run.s * p.F + c, left - j * STEP, db[j]);
                        } else {
                            if (p.dweight) store_weights<T, A, G>(slot_sums, true, c, left - j * STEP, dw[j]);
                            if (p.dbias) store_weights<T, A, G>(slot_sums, true, p.F + c, left - j * STEP, db[j]);
                        }
                    }
                } else {
                    constexpr int WIDE = G < 32 ? 32 : G, PARTS = NT / WIDE;
                    float* own = shared_sums + threadIdx.x / WIDE * 2 * a.tile;
                    __syncthreads();
                    if (threadIdx.x % WIDE < G) {
#pragma unroll
                        for (int j = 0; j < PER; ++j)
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const int c = t * P::NEXT + j * STEP + i * P::STEP;
                                if (c >= a.tile) continue;
                                own[c] = i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x;
                                own[a.tile + c] = i % 2 ? db[j][i / 2].y : db[j][i / 2].x;
                            }
                    }
                    __syncthreads();
                    for (int i = threadIdx.x; i < 2 * a.tile; i += NT) {
                        const int which = i >= a.tile, c = col0 + i - which * a.tile;
                        if (c >= F) continue;
                        float v = 0.0f;
#pragma unroll
                        for (int q = 0; q < PARTS; ++q) v += shared_sums[q * 2 * a.tile + i];
                        put(which, c, v);
                    }
                }
            }
            from = run_end;
            if (from >= n) break;
            run = run_of(p, c0 + from, run.s);
            begin();
            if (from >= end) break;
        }
        po += U * nexto;
        if constexpr (!KEEP) values_read();
    }
    if (want_dw && a.clear) clear_empty(p, col0, min(col0 + a.tile, F));
}

// Adds the parts of a segment that more than one chunk has rows of: blockIdx.x
// names the segment, or (by_start) the chunk in which it starts; blockIdx.y the
// first `lanes` x V of the sums that are wanted.  Each of the block's ADD_THREADS / lanes rows
// of threads adds an equal share of the parts in order, then theirs are added.
constexpr int ADD_THREADS = 512;
template <int V>
__global__ void __launch_bounds__(ADD_THREADS) norm_add_kernel(const __grid_constant__ GradArgs a, int by_start, int lanes) {
    __shared__ float sums[V][ADD_THREADS];
    const NormParams& p = a.p;
    int64_t s = blockIdx.x, begin = 0, end = p.R;
    if (by_start) {
        const Run run = run_of(p, min((int64_t(blockIdx.x) + 1) * a.chunk, p.R) - 1);
        s = run.s, begin = run.begin, end = run.end;
        if (s < 0 || begin / a.chunk != blockIdx.x) end = begin;
    } else if (p.offsets) {
        begin = offset_at(p, s), end = offset_at(p, s + 1);
    }
    // by every block, also one without work: what follows this kernel in the stream
    // may rely on the backward pass too
    grid_wait();
    if (begin >= end) return;
    const int64_t first = begin / a.chunk, last = (end - 1) / a.chunk;
    if (first == last) return;
    const int lane = threadIdx.x % lanes, share = threadIdx.x / lanes, shares = ADD_THREADS / lanes;
    const int parts = static_cast<int>(last - first + 1), each = (parts + shares - 1) / shares;
    const int q0 = share * each, q1 = min(q0 + each, parts);
    const int64_t i_end = p.dbias ? 2 * p.F : p.F;
    for (int64_t i0 = (p.dweight ? 0 : p.F) + int64_t(blockIdx.y) * lanes * V; i0 < i_end; i0 += int64_t(gridDim.y) * lanes * V) {
        const int64_t i = i0 + lane * V;
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = 0.0f;
        if (i < i_end) {
#pragma unroll 8
            for (int q = q0; q < q1; ++q) {
                const float* from = a.partials + (2 * (first + q) + (q == 0 ? 1 : 0)) * 2 * p.F + i;
                if constexpr (V == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(from));
                    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                } else {
                    v[0] += __ldcg(from);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) sums[k][threadIdx.x] = v[k];
        __syncthreads();
        for (int k = threadIdx.x; k < lanes * V; k += ADD_THREADS) {
            const int64_t c = i0 + k;
            if (c >= i_end) break;
            float total = 0.0f;
            for (int q = 0; q < shares; ++q) total += sums[k % V][q * lanes + k / V];
            void* out = c < p.F ? p.dweight : p.dbias;
            store_weight(out, p.weight_type, s * p.F + (c < p.F ? c : c - p.F), total);
        }
        __syncthreads();
    }
}

// Bytes of sums that a block of the backward pass may have to clear; above, a
// kernel of its own does (one row in 200 segments of 16,384 float32 columns, 26 MB:
// 408 us by the row's block, 31 so; 10 rows in 1,000,000 of 64, 512 MB: 5,750 and
// 102; one in 20 of 1,000, 160 KB: 16.4 and 14.4; two in 8 of 4,096, 128 KB a block:
// 14.9 and 16.4, one more launch).
constexpr int64_t CLEAR_SHARE = 64 * 1024;

int64_t ceil_to(int64_t n, int64_t d) { return (n + d - 1) / d; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Allows a kernel its shared memory: once per device (the call takes as long as
// a launch).  Callers hold the library's lock.
template <class K>
cudaError_t allow_smem(K* kernel, int bytes, int (&allowed)[64]) {
    if (bytes <= 40 * 1024) return cudaSuccess;      // (48 KB are allowed unasked, with the kernel's own)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || allowed[dev] >= bytes) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) allowed[dev] = bytes;
    return e;
}

template <class T, bool A, int G, int PER>
cudaError_t launch_rows(const NormParams& p, const NormPlan& plan, cudaStream_t stream) {
    constexpr int NT = G > 256 ? G : 256, U = forward_rows(A, sizeof(T), NT, PER), smem = Ring<T, A, G, PER, U, NT>::BYTES;
    auto* kernel = norm_kernel<T, A, G, PER, U, NT>;
    static int allowed[64] = {};
    const cudaError_t e = allow_smem(kernel, smem, allowed);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(plan.chunks), NT, smem, stream>>>(p, plan.chunk);
    return cudaGetLastError();
}

template <class T, bool A, int G, int PER>
cudaError_t launch_grad_rows(const GradArgs& a, const NormPlan& plan, cudaStream_t stream) {
    constexpr int NT = G > 256 ? G : 256, U = grad_rows(PER);
    auto* kernel = norm_grad_kernel<T, A, G, PER, U, NT>;
    const int smem = Ring<T, A, G, PER, 2 * U, NT>::BYTES + (G < NT ? NT / std::max(G, 32) * 2 * a.tile * 4 : 0);
    static int allowed[64] = {};
    const cudaError_t e = allow_smem(kernel, smem, allowed);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(static_cast<unsigned>(plan.chunks), plan.tiles), NT, smem, stream>>>(a);
    return cudaGetLastError();
}

// f(shape) for the shape of a plan, as constants: whether rows are aligned, threads of a row, packs of a thread.
template <bool ALIGNED, int GROUP, int PER> struct Shape {
    static constexpr bool aligned = ALIGNED;
    static constexpr int group = GROUP, per = PER;
};
template <class T, class F>
cudaError_t with_shape(const NormPlan& plan, F f) {
    constexpr int MOST = ROW_VALUES * sizeof(T) / 16;
#define SEG_NORM_SHAPE(a, g, n) \
    if (plan.aligned == a && plan.group == g && plan.per == n) return f(Shape<a, g, n>())
    SEG_NORM_SHAPE(true, 256, 1);
#define SEG_NORM_SHAPES(a)                    \
    SEG_NORM_SHAPE(a, 8, 1);                  \
    SEG_NORM_SHAPE(a, 8, MOST);               \
    SEG_NORM_SHAPE(a, 16, MOST);              \
    SEG_NORM_SHAPE(a, 32, MOST);              \
    SEG_NORM_SHAPE(a, 64, MOST);              \
    SEG_NORM_SHAPE(a, 128, MOST);             \
    SEG_NORM_SHAPE(a, 256, MOST);             \
    SEG_NORM_SHAPE(a, 512, MOST);             \
    SEG_NORM_SHAPE(a, 512, 2 * MOST);         \
    SEG_NORM_SHAPE(a, 1024, MOST);            \
    if constexpr (MOST == 4) SEG_NORM_SHAPE(a, 8, 2)
    SEG_NORM_SHAPES(true);
    SEG_NORM_SHAPES(false);
#undef SEG_NORM_SHAPES
#undef SEG_NORM_SHAPE
    return cudaErrorInvalidConfiguration;
}

template <class T>
cudaError_t launch_type(const NormParams& p, const NormPlan& plan, cudaStream_t stream) {
    if (plan.per == 0 && plan.aligned && plan.group == WIDE_THREADS) {
        static int allowed[64] = {};
        const int smem = static_cast<int>(WIDE_SLOTS * p.F * sizeof(T));
        const cudaError_t e = allow_smem(norm_wide_kernel<T>, smem, allowed);
        if (e != cudaSuccess) return e;
        norm_wide_kernel<T><<<static_cast<unsigned>(plan.chunks), WIDE_THREADS, smem, stream>>>(p, plan.chunk);
        return cudaGetLastError();
    }
    if (plan.per == 0) {
        norm_long_kernel<T><<<static_cast<unsigned>(plan.chunks), 256, 0, stream>>>(p);
        return cudaGetLastError();
    }
    return with_shape<T>(plan, [&](auto s) {
        if constexpr (s.group == 1024) return cudaErrorInvalidConfiguration;      // (wide rows: above)
        else return launch_rows<T, s.aligned, s.group, s.per>(p, plan, stream);
    });
}

template <class T>
cudaError_t launch_grad_type(const GradArgs& a, const NormPlan& plan, cudaStream_t stream) {
    if (a.sums) {
        norm_sums_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(a.p.R, int64_t(a.p.sms) * 8)), 256, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return with_shape<T>(plan, [&](auto s) {
        constexpr bool twice = s.per * static_cast<int>(16 / sizeof(T)) > ROW_VALUES;
        if constexpr (twice && (sizeof(T) == 4 || !s.aligned)) return cudaErrorInvalidConfiguration;
        else return launch_grad_rows<T, s.aligned, s.group, s.per>(a, plan, stream);
    });
}

}  // namespace

NormPlan plan_norm(bool grad, const NormParams& p) {
    NormPlan d{};
    const int size = p.type == PT_F32 ? 4 : 2, v = 16 / size;
    // whole 16-byte loads of every operand
    const bool vec = p.F % v == 0 && p.ldx % v == 0 && aligned16(p.x) && (!p.out || (p.ldo % v == 0 && aligned16(p.out))) &&
                     (!grad || (p.ldy % v == 0 && aligned16(p.dy))) && aligned16(p.weight) && aligned16(p.bias) && aligned16(p.dweight) && aligned16(p.dbias);
    d.aligned = vec;
    d.tiles = 1;
    const int64_t loads = ceil_to(p.F, v);
    const int most = ROW_VALUES / v;
    // as few threads for a row as hold it; where there are few rows, a block's, so
    // that each is over sooner
    if (p.R <= p.sms && loads > 32) {
        d.group = loads <= 256 * most ? 256 : loads <= 512 * most ? 512 : 1024;
    } else {
        d.group = 8;
        while (d.group < 1024 && int64_t(d.group) * most < loads) d.group *= 2;
    }
    // forward, as many again of a thread: 5,000 x 9,000 bfloat16 43 us, by 1,024
    // threads, which have no registers for the weights, 82.  Backward, aligned 16-bit
    // rows alone: 5,000 x 12,288 bfloat16 124 us, by 1,024 threads 137; float32, whose
    // ring does not hold two rows, 235 and 179; 5,000 x 9,001 bfloat16 288 and 237.
    const bool twice = d.group == 1024 && loads <= 1024 * most && (!grad || (vec && size == 2));
    if (twice) d.group = 512;
    d.threads = std::max(d.group, 256);
    const int64_t per = ceil_to(loads, d.group);
    d.per = twice ? 2 * most : most;
    if (d.group == 8 && per <= 2) d.per = static_cast<int32_t>(per);
    if (vec && d.group == 256 && per == 1) d.per = 1;
    // Wider rows, forward: from shared memory, or read again (5,000 x 9,001 bfloat16,
    // which registers hold, so 114 us and 73).
    const int64_t ring = WIDE_SLOTS * p.F * size;
    const bool from_ring = !grad && vec && loads > 1024 * most && ring <= 216 * 1024;
    if (from_ring || (!grad && d.group == 1024)) {
        d.per = 0;
        d.threads = d.group = from_ring ? WIDE_THREADS : 256;
    } else if (per > d.per) {
        if (grad) {
            d.tiles = static_cast<int32_t>(ceil_to(per, most));
            d.sums_bytes = ceil_to(p.R * 8, 256) * 256;
        }
    }
    const int rows = grad ? grad_rows(d.per) : forward_rows(vec, size, d.threads, d.per);
    const int64_t window = d.per == 0 ? 1 : d.threads / d.group * rows;
    const int64_t most_blocks = from_ring ? int64_t(p.sms) * (ring <= 108 * 1024 ? 2 : 1)
                                : d.per == 0 ? int64_t(p.sms) * 8
                                             : std::max<int64_t>(p.sms * resident(d.threads, d.per * v * (grad ? 2 * rows + 3 : rows + 2)) / d.tiles, 1);
    const int64_t least = ceil_to(p.R, most_blocks);
    d.chunk = ceil_to(least, window) * window;
    // backward, a block takes its runs one after the other: four of them on average
    // where that leaves part of a window (30 rows in 58 segments, both passes 44 -> 19 us)
    if (grad && p.S > 1) d.chunk = std::min(d.chunk, std::max(least, 4 * ceil_to(p.R, p.S)));
    d.chunks = ceil_to(p.R, d.chunk);
    if (d.per == 0 && !from_ring) d.chunks = std::min<int64_t>(p.R, most_blocks);
    if (grad) d.partial_bytes = ceil_to(d.chunks * 4 * p.F * 4, 256) * 256;
    // Each of the blocks that the rows need clears its share of the segments without
    // rows, whose sums may be nearly all that there is to store.
    if (grad && p.offsets) {
        const int64_t bytes = p.S * p.F * (p.weight_type == PT_F32 ? 4 : 2) * ((p.dweight ? 1 : 0) + (p.dbias ? 1 : 0));
        if (bytes > d.chunks * d.tiles * CLEAR_SHARE)
            d.clear_blocks = static_cast<int32_t>(std::min<int64_t>(ceil_to(ceil_to(p.S, 32) * ceil_to(p.F, CLEAR_COLUMNS), 8), int64_t(p.sms) * 8));
    }
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
    a.tile = static_cast<int32_t>(std::min<int64_t>(p.F, int64_t(plan.group) * plan.per * (p.type == PT_F32 ? 4 : 8)));
    a.chunk = plan.chunk;
    a.clear = p.offsets && (p.dweight || p.dbias) && plan.clear_blocks == 0;
    a.sums = plan.sums_for(p) > 0 ? reinterpret_cast<float*>(p.ws) : nullptr;
    a.partials = reinterpret_cast<float*>(p.ws + plan.sums_for(p));
    cudaError_t e;
    if (plan.clear_blocks > 0) {
        const int size = p.weight_type == PT_F32 ? 4 : 2;
        norm_clear_kernel<<<static_cast<unsigned>(plan.clear_blocks), 256, 0, stream>>>(p, size, p.F * size % 16 == 0 && aligned16(p.dweight) && aligned16(p.dbias));
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (p.type == PT_F32) e = launch_grad_type<float>(a, plan, stream);
    else if (p.type == PT_F16) e = launch_grad_type<__half>(a, plan, stream);
    else e = launch_grad_type<__nv_bfloat16>(a, plan, stream);
    if (e != cudaSuccess || plan.chunks < 2 || (!p.dweight && !p.dbias)) return e;
    const bool by_start = p.S >= plan.chunks;
    // the fewer segments, the more parts there are of each; four shares at least, for
    // segments of uneven lengths (20,011 rows in 64 of them: the two passes 73 us
    // with one share, 67 so)
    int shares = 4;
    while (shares < 32 && (plan.chunks / p.S + 1) / (shares * 2) >= 4) shares *= 2;
    const int lanes = ADD_THREADS / shares, v = p.F % 4 == 0 || (p.F % 2 == 0 && p.dweight && p.dbias) ? 4 : 1;      // (four sums of one kind, or of both)
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(by_start ? plan.chunks - 1 : p.S), static_cast<unsigned>(std::min<int64_t>(ceil_to(p.dweight && p.dbias ? 2 * p.F : p.F, lanes * v), 16384)));
    cfg.blockDim = dim3(ADD_THREADS);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, v == 4 ? norm_add_kernel<4> : norm_add_kernel<1>, a, static_cast<int>(by_start), lanes);
}

}  // namespace segred

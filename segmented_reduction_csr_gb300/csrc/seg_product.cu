// seg_product.cu -- products over the rows of segments (see seg_product.cuh)
// on the tensor cores (tcgen05, accumulators in tensor memory).
//
// One kernel serves all of them.  A tile is D[m, n] with m (128 lanes
// of tensor memory, 256 for a pair of CTAs) along the output's contiguous
// dimension and n (its columns, up to NT) along the other one:
//   forward, adapters  m: output columns, n: rows of one segment, sum over K;
//   weights            m: columns of dy,  n: columns of x,        sum over rows;
//   gated              m: 64 columns of the gate and the same 64 of the other
//                      projection, n: rows of one segment, sum over K.
// With the rows of a segment on n, whose extent an MMA takes in steps of 16,
// a ragged tail or a single row costs 16 columns, not a whole 128-row tile;
// and a warp's 32 lanes are 32 neighbouring output columns, so results leave
// coalesced whatever the alignment.
//
// Roles per CTA (persistent, one CTA per SM, tiles dealt round robin): two
// elected threads copy operands (tensor copies) into a ring of shared-memory
// stages, 64 steps of the sum each, rows of 128 bytes, swizzled; one thread
// issues the MMAs; eight warps drain one of two accumulators while the other
// fills.  Further warps where there is need: one that zeroes the rows of a
// weights' sum past the segment's end; eight that split float32; four that lay
// out the adapters' part.  Every wait has a time limit; a role that gives up
// says so in the device status word and all leave.
//
// What bounds it (gated: below, at its drain; GB300; measured peaks 6,793 GB/s, and 1,892 TFLOP/s in short
// runs, 1,706 held).  Times are of a call in a replayed graph / of calls back to
// back from Python:
//   training shapes: the tensor cores' clock and power.  32,768 rows, 32
//     segments, 2,048 x 4,096 bfloat16: forward 309-328 / 371 us = 1,676-1,781 /
//     1,482 TFLOP/s, weights 364-370 / 403 us;
//   decode: reading the matrices.  128 rows over 64 matrices of 2,048 x 1,024:
//     35 / 37 us = 6.6 TB/s of the matrices that are used;
//   single tokens: launch, one round trip to memory and the parts' exchange,
//     9 / 14 us for 2 rows and two 2,048 x 2,048 matrices (the host: 14);
//   float32: no unit alone.  Every value is in shared memory as float32 and as
//     parts, and the part products read those again, so a part of one operand
//     takes as many parts of the other at once as the accumulators have room
//     for.  1,000,000 x 64 times 64 x 64 in 50 segments: 105-116 / 109 us = 4.9
//     TB/s; the shared memory's data path is busy for 61 % of the time (warps 26,
//     operands of the MMAs 35), DRAM for 55.  Its weights' gradient, 149 / 152
//     us: 66 % (37 and 29), DRAM 47, and SMs that wait for the longest share, 22.
//
// float32: every value is split into three bfloat16 parts by truncation (8 + 8
// + 8 bits, exact) and six of the nine part products are accumulated; the
// other three are below 2^-21 of the whole each.
// The tensor cores cut what an addition shifts out of the accumulator: a sum of
// one sign loses about 2^-23.4 of it per 16 steps of full products, less while
// short products still fit (measured).  So for float32 the five small part
// products have accumulators of their own, and where the result is float32 the
// accumulators are added to it, rounded, every 512 (float32) or 768 (16-bit
// operands) steps: a sum of one sign is then low by 0.8e-6 (float32; 1.9e-6 where
// a part of 1,024 steps is not flushed), 1.3e-6 (bfloat16) or 4.4e-6 (float16).
// 16-bit results: LONGEST.
// Long sums with few tiles are cut into parts, added in order.  Forward: the
// parts of a tile are a cluster and add through its shared memory.  Weights,
// whose segments can have hundreds of parts: float32 partials in scratch, and
// a second kernel adds them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "seg_act.cuh"
#include "seg_common.cuh"
#include "seg_product.cuh"
#include "tc.cuh"

namespace segred {
namespace {

constexpr int KB = 64;                    // steps of the sum per stage: 128-byte rows of 16-bit values
constexpr int MT = 128;                   // lanes of a tile
constexpr int NEAR_SEGMENTS = 1024;       // up to here every CTA keeps the offsets in shared memory
constexpr int EPI_WARP = 4, EPW = 8;      // drain warps: their index mod 4 names their lanes, and the two of a quarter take turns at the columns
constexpr int LOAD_WARP = 12, LOADERS = 256;    // loader warps start here; their threads
constexpr int LOW_WARP = 12;              // four warps that lay out the adapters' part for the tensor cores
template <int MODE, bool TENSOR, int PL>
constexpr int threads_of() { return TENSOR && PL == 1 ? (MODE == PRODUCT_ADAPTERS ? 512 : 384) : 640; }
// Rows of a tile per run of rows with one adapter from which on the tile's
// low-rank part goes to the tensor cores (an MMA takes 16 columns at least;
// a run costs them a pass over the whole tile).
constexpr int LOW_RUN = 16;
constexpr int LOW_EVERY = 10;             // blocks of the sum between two of the low-rank part: about the time one takes to lay out
constexpr int LOW_TILES = 4;              // barriers of tiles whose low-rank part is done: three can be before the first of them has been drained
constexpr int NEVER_FLUSH = 1 << 28;         // more blocks than any sum has
// Steps that 16-bit results and the adapters' inner products sum up in one
// accumulator.  Its additions cut what they shift out, less than 2^-23 of it
// twice per 16 steps: 2^-11 of a sum of one sign at most (2e-4 measured at this
// length; 1,048,576 steps were off by 6e-3), which a float16 result's own
// rounding covers.  Longer sums are added up from pieces, rounded, in float32.
constexpr int64_t LONGEST = 32768;
constexpr int FLUSH_F32 = 8;              // blocks of a float32 sum in one accumulator
constexpr unsigned STATUS_PRODUCT_TIMEOUT = 8u;

// Stage ring of a kernel shape: PL 16-bit planes per operand, CG CTAs that share a tile.
template <int MODE, int NT, int PL, int CG, bool TENSOR>
struct Ring {
    static constexpr bool LOW = MODE == PRODUCT_ADAPTERS && TENSOR && PL == 1;   // a stage of its own for the low-rank part
    static constexpr int A_PLANE = MT * 128, B_PLANE = NT / CG * 128;
    static constexpr int STAGE = PL * (A_PLANE + B_PLANE);
    // (the loaders' plain loads are tracked in the L1 that shared memory leaves)
    static constexpr bool GATED = MODE == PRODUCT_GATED;
    static constexpr int ALL_STAGES = std::min(8, (PL == 3 ? (GATED ? 204800 : 221184) : TENSOR ? 200704 : 98304) / STAGE);
    static constexpr int STAGES = ALL_STAGES - (LOW ? 1 : 0);
    static constexpr bool ROW3 = PL == 3 && NT == 64;            // a part of A times several parts of B at once
    static constexpr int ACC = PL == 1 ? NT : 256;               // tensor-memory columns of one accumulator
    static constexpr int BARS = 3 * STAGES + 7 + LOW_TILES;
    // the drain warps' staging; PL == 3 keeps it (adapters alone need it there) in the space of the offsets
    static constexpr int STAGING = PL == 1 || GATED ? 2048 : 1024;
    static constexpr int STAGED = PL == 1 || GATED ? EPW * STAGING : 0;
    static constexpr int NEAR = 2 * (NEAR_SEGMENTS + 1) * 4;
    static_assert(NEAR >= EPW * 1024, "room for that staging");
    static constexpr int SMEM = ALL_STAGES * STAGE + STAGED + NEAR + BARS * 8 + 128 + NT * 4 * (LOW ? 2 : 1) + 1024;   // 1024: alignment of the stages
    static_assert(SMEM <= 232448, "shared memory of an SM");
};

struct KernelArgs {
    ProductParams p;
    int32_t mtiles, ntiles, parts, part_blocks, kblocks;
    int32_t box_rows;   // rows of one copy of x
    int32_t a_rows;     // rows of one copy of A whose sum is contiguous
    int32_t twin;       // at most 64 lanes, laid out twice: the drain warps of the second 64 share the first's work
    int32_t wide_rows;  // 16-bit results: 16-byte stores fit
    int32_t wide_pre;   // the same of gated's 16-bit products
    int32_t flush;      // blocks of the sum after which the accumulators go to the result
    int32_t add_by_start;
    int64_t half_w;     // gated: elements from the gate's columns of a matrix to the other projection's
    int64_t chunk, row_tiles, cols_m, cols_n;   // cols_*: extent of the tile dimensions (forward: cols_n unused)
    int* far;          // offsets and tile prefix of more than NEAR_SEGMENTS segments
    float* partials;
};

__device__ __forceinline__ int offset_at(const ProductParams& p, int64_t s) {
    const int64_t o = p.off64 ? __ldg(static_cast<const int64_t*>(p.offsets) + s)
                              : static_cast<int64_t>(__ldg(static_cast<const uint32_t*>(p.offsets) + s));
    return static_cast<int>(clamp_off(o, p.R));
}

// Tiles of rows (forward) or parts of the rows (weights) of segment s.
template <int MODE, int NT>
__device__ __forceinline__ int segment_items(const KernelArgs& a, int64_t s, int b, int e) {
    const int len = e > b ? e - b : 0;
    if (MODE == PRODUCT_WEIGHTS) return len == 0 ? 1 : static_cast<int>((len + a.chunk - 1) / a.chunk);
    if (a.p.index) {
        const int l = __ldg(a.p.index + s);
        if (l < 0 || l >= a.p.L) return 0;
    }
    return (len + NT - 1) / NT;
}

// beg[s] = offset s, pre[s] = items of the segments before s (s = 0 .. S), by
// all threads of the CTA, PER segments a thread at a time.
template <int MODE, int NT, int PER>
__device__ void fill_prefix(const KernelArgs& a, int* beg, int* pre) {
    __shared__ int64_t warp_sum[32];
    __shared__ int64_t carry;
    const int t = threadIdx.x, nth = blockDim.x, lane = t & 31, warp = t >> 5;
    const int64_t S = a.p.S;
    if (t == 0) carry = 0;
    for (int64_t s = t; s <= S; s += nth) beg[s] = offset_at(a.p, s);
    __syncthreads();
    for (int64_t s0 = 0; s0 < S; s0 += nth * PER) {
        const int64_t s = s0 + t * PER;
        int v[PER];
        int64_t own = 0;   // 64 bits: offsets that go back and forth add up to more than the rows
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = s + i < S ? segment_items<MODE, NT>(a, s + i, beg[s + i], beg[s + i + 1]) : 0;
            own += v[i];
        }
        int64_t x = own;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        int64_t before = carry + x - own;
        for (int w = 0; w < warp; ++w) before += warp_sum[w];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (s + i < S) pre[s + i] = static_cast<int>(min(before, int64_t(INT_MAX)));
            before += v[i];
        }
        __syncthreads();
        if (t == nth - 1) carry = before;
        __syncthreads();
    }
    if (t == 0) pre[S] = static_cast<int>(min(carry, int64_t(INT_MAX)));
    __syncthreads();
}

// The offsets and prefix of many segments, once per call.
template <int MODE, int NT>
__global__ void __launch_bounds__(1024) prefix_kernel(const __grid_constant__ KernelArgs a) {
    fill_prefix<MODE, NT, 8>(a, a.far, a.far + a.p.S + 1);
}

struct Item {
    int seg = 0;
    int each_of = -1, each = 0;      // forward: rows of a tile of segment each_of
    int row0, rows;     // forward: the tile's rows; weights: the rows it sums over
    int m0, n0;
    int kb0, kb1;       // 64-wide blocks of the sum
    int part, parts;
    int64_t slot;
};

// Item i; `t` holds the item before it (seg 0 at the start): a CTA's items
// come in order, so its segments are found by going on from there.
template <int MODE, int NT, int CG>
__device__ __forceinline__ void item_at(const KernelArgs& a, const int* beg, const int* pre, uint32_t i, Item& t) {
    int q;
    constexpr int LANES = MODE == PRODUCT_GATED ? MT / 2 : MT;      // columns of the result that a CTA's tile has
    const uint32_t mtiles = a.mtiles;
    if (MODE == PRODUCT_WEIGHTS) {
        const uint32_t per = mtiles * a.ntiles, r = i % per;
        q = static_cast<int>(i / per);
        t.m0 = static_cast<int>(r % mtiles) * (MT * CG);
        t.n0 = static_cast<int>(r / mtiles) * NT;
    } else {
        const uint32_t tile = a.parts > 1 ? i / a.parts : i;
        t.part = static_cast<int>(i - tile * a.parts);
        q = static_cast<int>(mtiles > 1 ? tile / mtiles : tile);
        t.m0 = static_cast<int>(tile - q * mtiles) * (LANES * CG);
        t.n0 = 0;
    }
    int b = 0, e = static_cast<int>(a.p.R), first = 0, count;
    if (MODE == PRODUCT_ADAPTERS) {
        t.seg = 0;
        count = static_cast<int>(a.row_tiles);
    } else {
        int lo = t.seg;                             // the last segment whose items start at or before q
        for (int k = 0; k < 4 && pre[lo + 1] <= q; ++k) ++lo;
        if (pre[lo + 1] <= q) {
            int hi = static_cast<int>(a.p.S);
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid] <= q) lo = mid; else hi = mid;
            }
        }
        t.seg = lo;
        b = beg[lo];
        e = beg[lo + 1];
        first = pre[lo];
        count = pre[lo + 1] - first;
    }
    const int len = e > b ? e - b : 0, j = q - first;
    if (MODE == PRODUCT_WEIGHTS) {
        const int64_t at = j * a.chunk;
        t.row0 = static_cast<int>(b + at);
        t.rows = static_cast<int>(len - at < a.chunk ? len - at : a.chunk);
        t.kb0 = 0;
        t.kb1 = (t.rows + KB - 1) / KB;
        t.part = j;
        t.parts = count;
        // parts of one split segment start `chunk` rows apart, and a block of
        // `chunk` rows holds the starts of at most two split segments' parts,
        // one of them a first part: so these numbers are each used once
        const int per = a.mtiles * a.ntiles, r = t.m0 / (MT * CG) + t.n0 / NT * a.mtiles;
        t.slot = (2 * (t.row0 / a.chunk) + (j == 0 ? 1 : 0)) * per + r;
    } else {
        // the segment's rows in equal tiles of a multiple of 16
        if (t.each_of != t.seg) {
            t.each_of = t.seg;
            t.each = ((len + count - 1) / count + 15) & ~15;
            t.each = t.each < NT ? t.each : NT;
        }
        const int each = t.each;
        t.row0 = b + j * each;
        t.rows = len - j * each < each ? len - j * each : each;
        t.kb0 = t.part * a.part_blocks;
        t.kb1 = min(t.kb0 + a.part_blocks, a.kblocks);
        t.parts = a.parts;
        t.slot = 0;
    }
}

__device__ __forceinline__ void bar_drain() { asm volatile("bar.sync 1, %0;" ::"n"(EPW * 32) : "memory"); }
// The same, and whether `ok` holds in all the drain warps: they give up together or not at all.
__device__ __forceinline__ bool bar_drain_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u), "n"(EPW * 32)
        : "memory");
    return r != 0;
}
// In how many of the drain warps' threads `yes` holds.
__device__ __forceinline__ int bar_drain_count(bool yes) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.popc.u32 %0, 1, %2, p;\n\t}"
        : "=r"(r)
        : "r"(yes ? 1u : 0u), "n"(EPW * 32)
        : "memory");
    return r;
}
// The four low-rank warps, as bar_drain and bar_drain_all.
__device__ __forceinline__ void bar_low() { asm volatile("bar.sync 2, 128;" ::: "memory"); }
__device__ __forceinline__ bool bar_low_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u)
        : "memory");
    return r != 0;
}

// The adapter of a row: its segment's, or -1.  near: the offsets and then the adapters in shared memory, or NULL.
__device__ __forceinline__ int adapter_of(const ProductParams& p, const int* near, int row) {
    auto offset = [&](int64_t s) { return near ? near[s] : offset_at(p, s); };
    int64_t lo = 0, hi = p.S;      // the last segment that starts at or before the row
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (offset(mid) <= row) lo = mid; else hi = mid;
    }
    int l = -1;
    if (p.S > 0 && offset(lo) <= row && row < offset(lo + 1)) l = near ? near[NEAR_SEGMENTS + 1 + lo] : __ldg(p.index + lo);
    return l >= 0 && l < p.L ? l : -1;
}

// A bounded wait; CG == 2: for arrivals of both CTAs.  The clock is read only
// after a few hundred tries: a read takes longer than a stage does.
template <int CG>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, unsigned int* status) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (CG == 2 ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((i & 255) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > WAIT_LIMIT_NS) break;
        }
    }
    atomicOr(status, STATUS_PRODUCT_TIMEOUT);
    return false;
}
// The same for a whole warp.
template <int CG>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned int* status) {
    return __all_sync(0xffffffffu, wait_for<CG>(bar, parity, status));
}

// Value i of every lane to row i of `out`, rows `step` apart, for i < n.
template <class T, int W, class F>
__device__ __forceinline__ void store_rows(T* out, int64_t step, const float (&v)[W], int n, F narrow) {
    if (n >= W) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            T* o = out + i * step;
            o[0] = narrow(v[i]);
            o[step] = narrow(v[i + 1]);
            o[2 * step] = narrow(v[i + 2]);
            o[3 * step] = narrow(v[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i < n) out[i * step] = narrow(v[i]);
    }
}

__device__ __forceinline__ uint32_t narrow_pair(float a, float b, int type) {
    uint32_t r;
    if (type == PT_F16) asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    else asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

// W columns of the tile of this warp's 32 lanes to the result: `at` is lane
// 0's place in the first of n rows.  16-bit rows that allow it are turned in
// the warp's staging (rows of 64 bytes) and leave 16 bytes per thread: a
// store of 2 bytes per lane took 70 cycles a row.
template <int W>
__device__ __forceinline__ void store_result(const KernelArgs& a, int64_t at, int64_t step, const float (&v)[W], int n,
                                             int lanes, int lane, unsigned char* staging) {
    const int type = a.p.out_type;
    if (type == PT_F32) {
        if (lane < lanes) store_rows(static_cast<float*>(a.p.out) + at + lane, step, v, n, [](float x) { return x; });
        return;
    }
    if (!a.wide_rows) {
        if (lane >= lanes) return;
        uint16_t* o = static_cast<uint16_t*>(a.p.out) + at + lane;
        store_rows(o, step, v, n, [type](float x) { return static_cast<uint16_t>(narrow_pair(x, 0.0f, type)); });
        return;
    }
    uint16_t* s = reinterpret_cast<uint16_t*>(staging) + lane;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < W; i += 2) {
        const uint32_t two = narrow_pair(v[i], v[i + 1], type);
        s[i * 32] = static_cast<uint16_t>(two);
        s[i * 32 + 32] = static_cast<uint16_t>(two >> 16);
    }
    __syncwarp();
    const int unit = lane & 3;
    uint16_t* o = static_cast<uint16_t*>(a.p.out) + at + unit * 8;
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
        const int row = i * 8 + (lane >> 2);
        if (row < n && unit * 8 < lanes) *reinterpret_cast<uint4*>(o + row * step) = *reinterpret_cast<const uint4*>(staging + row * 64 + unit * 16);
    }
}

// This warp's columns of a finished tile, from tensor memory to 16-bit rows
// that take 16-byte stores: 32 columns at a time, in 8 x 8 blocks that the
// store to the warp's staging transposes (2-byte stores there, 32 a column
// group, took twice the time), its 16-byte units turned by the row against
// bank conflicts.
template <int STRIDE>
__device__ __forceinline__ void store_tile(const KernelArgs& a, uint32_t from, bool summed, int c, int columns, int64_t at, int64_t step,
                                           int lanes, int lane, unsigned char* staging) {
    const int type = a.p.out_type;
    float v[32];
    if (c < columns && summed) tmem_load_blocks(from + c, v);
    for (; c < columns; c += STRIDE) {
        uint32_t two[16];
        if (summed) {
            tmem_wait(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) two[i] = narrow_pair(v[2 * i], v[2 * i + 1], type);
            if (c + STRIDE < columns) tmem_load_blocks(from + c + STRIDE, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) two[i] = 0;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = 8 * k + (lane & 7);
            store_blocks_t(staging + row * 64 + (((lane >> 3) ^ (row >> 1 & 3)) << 4), two[2 * k], two[2 * k + 1], two[8 + 2 * k], two[8 + 2 * k + 1]);
        }
        __syncwarp();
        const int unit = lane & 3;
        uint16_t* o = static_cast<uint16_t*>(a.p.out) + at + c * step + unit * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + (lane >> 2);
            if (c + row < columns && unit * 8 < lanes)
                *reinterpret_cast<uint4*>(o + row * step) = *reinterpret_cast<const uint4*>(staging + row * 64 + ((unit ^ (row >> 1 & 3)) << 4));
        }
    }
}

// ---------------------------------------------------------------------------
// The gated block's drain.  Lanes 0 to 63 of a tile are the gate's columns, 64
// to 127 the other projection's, so what belongs together is in the lanes of
// two warps, `quarter` and `quarter` ^ 2.  Each of them takes half of the rows
// and gives the other half of its values to the other one, through shared
// memory: 2 x 64 KB a tile of 256 rows, under a tenth of what its MMAs read.
// 32,768 rows, 32 x (2,048 x 2,048 twice) bfloat16: 310 us, as the plain product
// of as many columns takes (312: clock and power), and 348 with the float32
// products kept; 4,161 uneven rows, 16 x (1,024 x 2,048 twice) float16 42 us (the
// plain product 39); 128 rows, 64 x (2,048 x 1,024 twice) bfloat16 59 us = 6.3 TB/s
// of the matrices in use.  Short sums are bound by the drain: 32,768 rows, 8 x (64 x
// 512 twice) bfloat16 35 us, of which twice the drain warps would save 4 and cost the
// long sums 1 %.
// (16 columns of each projection by turns in the lanes would need no exchange,
// but a matrix whose columns are contiguous cannot be copied so.)

// Lane's values of n rows `step` apart from element `at` of a tensor of any type.
template <int W>
__device__ __forceinline__ void store_any(void* out, int type, int64_t at, int64_t step, const float (&v)[W], int n) {
    if (type == PT_F32) store_rows(static_cast<float*>(out) + at, step, v, n, [](float x) { return x; });
    else store_rows(static_cast<uint16_t*>(out) + at, step, v, n, [type](float x) { return static_cast<uint16_t>(narrow_pair(x, 0.0f, type)); });
}

// f[i] = act(g(i)) * u(i), with the kind of activation outside of the loop, by
// the special function unit for float32 too: off by 4 + 1.2 |g| (silu, sigmoid), 4 +
// 4.2 |q| (gelu_tanh's q) or 23 + 0.85 g^2 (gelu) units of 2^-23 at most (see
// seg_act.cuh), where the products are by up to 2^-20 of their terms' sizes, and the
// drain warps' time is what bounds a float32 tile (expf and a division: 1,000,000 x
// 64 times 64 x 64 twice 262 us, so 166).
template <int W, class G, class U>
__device__ __forceinline__ void gate(int kind, float (&f)[W], G g, U u) {
    auto all = [&](auto k) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float slope;
            f[i] = activate<true, false>(k(), g(i), slope) * u(i);
        }
    };
    if (kind == ACT_SILU) all([] { return ACT_SILU; });
    else if (kind == ACT_GELU) all([] { return ACT_GELU; });
    else if (kind == ACT_GELU_TANH) all([] { return ACT_GELU_TANH; });
    else if (kind == ACT_RELU) all([] { return ACT_RELU; });
    else all([] { return ACT_SIGMOID; });
}

// Both warps of a pair; 3 .. 6 of the CTA's barriers.
__device__ __forceinline__ void bar_pair(int quarter, int group) { asm volatile("bar.sync %0, 64;" ::"r"(3 + group * 2 + (quarter & 1)) : "memory"); }

// From v's two halves (`low` and `high` name the registers): the results of this
// warp's half of the rows.  The two warps of a pair take different ways (a choice
// of registers for each value took a fifth of the drain's instructions).  TURNS:
// the caller takes two places of the staging in turns, so that the barrier before
// the next values are read is enough.
template <int W, bool TURNS, class Low, class High>
__device__ __forceinline__ void exchange_and_gate(int kind, const float (&v)[W], float (&f)[W / 2], Low low, High high, int lane, int quarter,
                                                  int group, unsigned char* own, int staging) {
    constexpr int H = W / 2;
    const bool second = quarter >= 2;
    float4* to = reinterpret_cast<float4*>(own) + lane;
    const float4* other = reinterpret_cast<const float4*>(second ? own - 2 * staging : own + 2 * staging) + lane;
    if (second) {
#pragma unroll
        for (int i = 0; i < H; i += 4) to[i * 8] = make_float4(v[low(i)], v[low(i + 1)], v[low(i + 2)], v[low(i + 3)]);
    } else {
#pragma unroll
        for (int i = 0; i < H; i += 4) to[i * 8] = make_float4(v[high(i)], v[high(i + 1)], v[high(i + 2)], v[high(i + 3)]);
    }
    bar_pair(quarter, group);
    float got[H];
#pragma unroll
    for (int i = 0; i < H; i += 4) {
        const float4 x = other[i * 8];
        got[i] = x.x, got[i + 1] = x.y, got[i + 2] = x.z, got[i + 3] = x.w;
    }
    if (!TURNS) bar_pair(quarter, group);      // the staging may be written again
    if (second) gate(kind, f, [&](int i) { return got[i]; }, [&](int i) { return v[high(i)]; });
    else gate(kind, f, [&](int i) { return v[low(i)]; }, [&](int i) { return got[i]; });
}

// W rows from row0 on, n of which there are, of this warp's lanes: register i holds row i.
template <bool TURNS, int W>
__device__ __forceinline__ void gate_rows(const KernelArgs& a, const float (&v)[W], int64_t row0, int n, int64_t m, int lanes, int lane,
                                          int quarter, int group, unsigned char* own, int staging) {
    const ProductParams& p = a.p;
    if (p.pre && lane < lanes) store_any(p.pre, p.pre_type, row0 * p.ldp + (quarter >> 1) * a.cols_m + m + lane, p.ldp, v, n);
    float f[W / 2];
    exchange_and_gate<W, TURNS>(p.activation, v, f, [](int i) { return i; }, [](int i) { return W / 2 + i; }, lane, quarter, group, own, staging);
    const int first = (quarter >> 1) * (W / 2);
    if (lane < lanes) store_any(p.out, p.out_type, (row0 + first) * p.ldo + m + lane, p.ldo, f, n - first);
}

// 16-bit results that take 16-byte stores, 32 rows at a time in 8 x 8 blocks as in
// store_tile; the next ones come from tensor memory while these are stored.
template <int STRIDE>
__device__ __forceinline__ void gate_blocks(const KernelArgs& a, uint32_t from, int64_t row0, int c, int columns, int64_t m, int lanes, int lane,
                                            int quarter, int group, unsigned char* own, int staging) {
    const ProductParams& p = a.p;
    const int half = quarter >> 1, unit = lane & 3;
    const bool wide = p.pre && p.pre_type == PT_F32;
    float v[32], rows[32];      // the sums in blocks; the same in rows of the lanes
    if (c < columns) {
        tmem_load_blocks(from + c, v);
        if (wide) tmem_load(from + c, rows);
    }
    for (; c < columns; c += STRIDE) {
        const int n = columns - c;
        tmem_wait(v);
        if (wide) {
            // (rows of 128 bytes, straight from the lanes)
            tmem_wait(rows);
            if (lane < lanes)
                store_rows(static_cast<float*>(p.pre) + (row0 + c) * p.ldp + half * a.cols_m + m + lane, p.ldp, rows, n, [](float x) { return x; });
        } else if (p.pre) {
            uint32_t two[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) two[i] = narrow_pair(v[2 * i], v[2 * i + 1], p.pre_type);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = 8 * k + (lane & 7);
                store_blocks_t(own + row * 64 + (((lane >> 3) ^ (row >> 1 & 3)) << 4), two[2 * k], two[2 * k + 1], two[8 + 2 * k], two[8 + 2 * k + 1]);
            }
            __syncwarp();
            uint16_t* o = static_cast<uint16_t*>(p.pre) + (row0 + c) * p.ldp + half * a.cols_m + m + unit * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i * 8 + (lane >> 2);
                if (row < n && unit * 8 < lanes) *reinterpret_cast<uint4*>(o + row * p.ldp) = *reinterpret_cast<const uint4*>(own + row * 64 + ((unit ^ (row >> 1 & 3)) << 4));
            }
            __syncwarp();
        }
        // registers 16 h + 4 k + 2 e + b of rows 8 k + ..: k = 0, 1 are the first 16 rows
        float f[16];
        exchange_and_gate<32, false>(p.activation, v, f, [](int i) { return (i & 7) + 2 * (i & 8); }, [](int i) { return (i & 7) + 2 * (i & 8) + 8; },
                                     lane, quarter, group, own, staging);
        if (c + STRIDE < columns) {
            tmem_load_blocks(from + c + STRIDE, v);
            if (wide) tmem_load(from + c + STRIDE, rows);
        }
        uint32_t two[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) two[i] = narrow_pair(f[2 * i], f[2 * i + 1], p.out_type);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = 8 * k + (lane & 7);
            store_blocks_t(own + row * 64 + (((lane >> 3) ^ (row >> 1 & 3)) << 4), two[2 * k], two[2 * k + 1], two[4 + 2 * k], two[4 + 2 * k + 1]);
        }
        __syncwarp();
        uint16_t* o = static_cast<uint16_t*>(p.out) + (row0 + c + half * 16) * p.ldo + m + unit * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = i * 8 + (lane >> 2);
            if (half * 16 + row < n && unit * 8 < lanes)
                *reinterpret_cast<uint4*>(o + row * p.ldo) = *reinterpret_cast<const uint4*>(own + row * 64 + ((unit ^ (row >> 1 & 3)) << 4));
        }
        __syncwarp();
    }
}

// W columns of a tile's sums in 32 lanes: of 16-bit operands, or the accumulators of float32 parts by size.
template <class R, int NT, int PL, int W>
__device__ __forceinline__ void load_sums(uint32_t from, float (&v)[W]) {
    if constexpr (PL > 1) {
        // (the small sums first)
        float mid[W], hi[W];
        tmem_load(from + NT, v);
        if constexpr (R::ROW3) tmem_load(from + 2 * NT, mid);
        tmem_load(from, hi);
        tmem_wait(v);
        if constexpr (R::ROW3) {
            tmem_wait(mid);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += mid[j];
        }
        tmem_wait(hi);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += hi[j];
    } else {
        tmem_load(from, v);
        tmem_wait(v);
    }
}

// ---------------------------------------------------------------------------

// The adapters' part of a tile, by the float32 pipes while the tensor cores
// work on: v[j] = sum_k u[row c + j, k] b[l_j, m, k] for 8 rows of this
// lane's column m at a time, 16 ranks a step.  The rows' u go through the
// warp's staging, b to the registers of the column's lane.  What a step needs
// is fetched during the step before; where the 8 rows have different
// adapters (a decode step), their b are fetched together at the step itself.
template <int PL, bool WIDE>
struct LowRank {
    static constexpr int SIZE = PL == 1 ? 2 : 4;
    static constexpr int WORDS = 16 * SIZE / 4;          // of 16 ranks
    static constexpr int AHEAD = WIDE ? 4 : 2;           // rows whose b are fetched together (as registers allow)
    const ProductParams& p;
    const int* tile_adapter;
    float4* su;                                          // [8 rows][4]
    int64_t m, stride;                                   // the lane's column; bytes from one adapter's b to the next
    int row0, rows, lane, rank;
    bool vec;
    // the next step
    float4 u;
    uint32_t b[WORDS];
    int mine, one;       // the adapter of row lane / 4; of all 8 rows, -1: none has one, -2: they differ

    __device__ __forceinline__ LowRank(const ProductParams& p_, const int* table, unsigned char* staging, int lane_)
        : p(p_), tile_adapter(table), su(reinterpret_cast<float4*>(staging)), lane(lane_), rank(static_cast<int>(p_.rank)) {
        stride = p.N * rank * SIZE;
        vec = rank * SIZE % 16 == 0 && (reinterpret_cast<uintptr_t>(p.b) & 15) == 0;
    }

    __device__ __forceinline__ void fetch_b(uint32_t (&r)[WORDS], int l, int q) const {
        const bool in = m < p.N && l >= 0;
        const int width = in ? rank - q : 0;
        const unsigned char* src = static_cast<const unsigned char*>(p.b) + (in ? l * stride + (m * rank + q) * SIZE : 0);
        if (vec) {       // predicated loads, no branch between those of several rows
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) {
                const uint4 x = k * 16 < width * SIZE ? __ldg(reinterpret_cast<const uint4*>(src) + k) : make_uint4(0, 0, 0, 0);
                r[4 * k] = x.x, r[4 * k + 1] = x.y, r[4 * k + 2] = x.z, r[4 * k + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < WORDS; ++k) r[k] = 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (k >= width) continue;
                if constexpr (PL == 1) r[k / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(src) + k)) << (k % 2 * 16);
                else r[k] = __ldg(reinterpret_cast<const uint32_t*>(src) + k);
            }
        }
    }

    __device__ __forceinline__ void fetch(int c, int q) {
        const int row = lane >> 2, unit = lane & 3, width = rank - q - unit * 4;
        if (q == 0) {
            mine = c + row < rows ? tile_adapter[c + row] : -1;
            const bool in = c + row < rows;
            const int l0 = __shfl_sync(0xffffffffu, mine, 0);
            one = __all_sync(0xffffffffu, !in || mine == l0) ? l0 : -2;
        }
        u = make_float4(0, 0, 0, 0);
        if (mine >= 0 && width > 0) {
            const float* src = p.u + (int64_t(row0) + c + row) * rank + q + unit * 4;
            if (rank % 4 == 0) {
                u = *reinterpret_cast<const float4*>(src);
            } else {
                u.x = src[0];
                if (width > 1) u.y = src[1];
                if (width > 2) u.z = src[2];
                if (width > 3) u.w = src[3];
            }
        }
        if (one >= 0) fetch_b(b, one, q);
    }

    __device__ __forceinline__ void begin(int row0_, int rows_, int64_t m_, int c) {
        row0 = row0_, rows = rows_, m = m_;
        if (c < rows) fetch(c, 0);
    }

    __device__ __forceinline__ void widen(float (&f)[16], const uint32_t (&r)[WORDS]) const {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if constexpr (PL == 3) f[k] = __uint_as_float(r[k]);
            else if (p.type == PT_BF16) f[k] = __uint_as_float(k % 2 ? r[k / 2] & 0xffff0000u : r[k / 2] << 16);
            else f[k] = __half2float(__ushort_as_half(static_cast<uint16_t>(k % 2 ? r[k / 2] >> 16 : r[k / 2])));
        }
    }

    __device__ __forceinline__ float dot(float s, int j, const float (&f)[16]) const {
        float s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = su[j * 4 + k];
            s = fmaf(x.x, f[4 * k], s);
            s2 = fmaf(x.y, f[4 * k + 1], s2);
            s = fmaf(x.z, f[4 * k + 2], s);
            s2 = fmaf(x.w, f[4 * k + 3], s2);
        }
        return s + s2;
    }

    // Rows c .. c + 7, fetched before; then rows `next` are.
    __device__ __forceinline__ void rows_of(float (&v)[8], int c, int next) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        for (int q = 0; q < rank; q += 16) {
            const int l_mine = mine, l_one = one;
            float f[16];
            __syncwarp();
            su[lane] = u;
            if (l_one >= 0) widen(f, b);
            __syncwarp();
            if (q + 16 < rank && l_one != -1) fetch(c, q + 16);
            else if (next < rows) fetch(next, 0);
            if (l_one == -1) return;
            if (l_one >= 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = dot(v[j], j, f);
                continue;
            }
#pragma unroll
            for (int j0 = 0; j0 < 8; j0 += AHEAD) {
                uint32_t raw[AHEAD][WORDS];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    fetch_b(raw[j], __shfl_sync(0xffffffffu, l_mine, (j0 + j) * 4), q);
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (__shfl_sync(0xffffffffu, l_mine, (j0 + j) * 4) < 0) continue;
                    widen(f, raw[j]);
                    v[j0 + j] = dot(v[j0 + j], j0 + j, f);
                }
            }
        }
    }
};

// ---------------------------------------------------------------------------
// The loader warps: blocks of a row-major matrix into 128-byte swizzled rows,
// zero outside [.., row_end) x [.., col_end).

// One operand of a stage: `rows` 128-byte rows of shared memory, 64 values
// each.  outer: every 64 rows are the block's 64 steps of the sum for the
// next 64 columns; else they are rows of the matrix.
struct Operand {
    const void* base;
    int64_t ld;
    int64_t row0, row_end;
    int64_t col0, col_end;
    int rows;
    bool outer;
    int steps;       // outer: of a block's 64 steps, those that are used (a multiple of 16)
};

// The three bfloat16 parts of two values: by truncation, each rest exact.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&r)[3]) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        r[k] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
        x -= __uint_as_float(r[k] << 16);
        y -= __uint_as_float(r[k] & 0xffff0000u);
    }
}

// float32 rows of 64 values that tensor copies left in the second (values 0
// to 31) and third plane, into their parts in all three.  A warp takes two
// whole rows at a time, four times over, and writes when all have been read.
__device__ __forceinline__ void split_rows(int rows, int valid, unsigned char* dst, int plane) {
    constexpr int STEP = LOADERS / 16, AHEAD = 4;
    const int t = threadIdx.x - LOAD_WARP * 32, q = t & 15, row = t >> 4;      // 16 bytes q of the row; 8 units of 8 values
    const unsigned char* from = dst + row * 128 + (1 + (q >> 3)) * plane + (((q & 7) ^ (row & 7)) << 4);
    unsigned char* to = dst + row * 128 + (((q >> 1) ^ (row & 7)) << 4) + (q & 1) * 8;
    for (int r = row; r - row < rows; r += AHEAD * STEP) {
        float4 x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (r - row + i * STEP < rows) x[i] = *reinterpret_cast<const float4*>(from + i * STEP * 128);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (r - row + i * STEP >= rows) break;
            if (((r + i * STEP) & 63) >= valid) x[i] = make_float4(0, 0, 0, 0);
            uint32_t a[3], b[3];
            split_pair(x[i].x, x[i].y, a);
            split_pair(x[i].z, x[i].w, b);
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(to + k * plane + i * STEP * 128) = make_uint2(a[k], b[k]);
        }
        from += AHEAD * STEP * 128;
        to += AHEAD * STEP * 128;
    }
}

// An operand of any alignment, by all loaders: 8 values of a row per thread,
// one by one (16-bit: in pairs where its rows allow that), the loads of two
// units together.
template <int PL>
__device__ __forceinline__ void load_any(const Operand& x, unsigned char* dst, int plane) {
    constexpr int AHEAD = 2;
    const int t = threadIdx.x - LOAD_WARP * 32, unit = t & 7;
    const bool pairs = PL == 1 && (reinterpret_cast<uintptr_t>(x.base) & 3) == 0 && x.ld % 2 == 0 && x.col_end % 2 == 0;
    const int count = x.outer ? (x.rows >> 6) * x.steps : x.rows;
    auto row_of = [&](int i) { return x.outer && x.steps < 64 ? i / x.steps * 64 + i % x.steps : i; };
    for (int row0 = t >> 3; row0 < count; row0 += AHEAD * LOADERS / 8) {
        uint32_t raw[AHEAD][8];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at_row = row0 + i * LOADERS / 8, row = at_row < count ? row_of(at_row) : x.rows;
            const int64_t r = x.row0 + (x.outer ? row & 63 : row), c = x.col0 + unit * 8 + (x.outer ? row & ~63 : 0);
            const bool in = row < x.rows && r < x.row_end;
            const int64_t at = r * x.ld + c;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (PL == 1) {
                    if (pairs) {
                        if (k < 4) raw[i][k] = in && c + 2 * k < x.col_end ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(x.base) + at) + k) : 0;
                    } else {
                        raw[i][k] = in && c + k < x.col_end ? __ldg(static_cast<const uint16_t*>(x.base) + at + k) : 0;
                    }
                } else {
                    raw[i][k] = in && c + k < x.col_end ? __ldg(static_cast<const uint32_t*>(x.base) + at + k) : 0;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (row0 + i * LOADERS / 8 >= count) break;
            const int row = row_of(row0 + i * LOADERS / 8);
            unsigned char* to = dst + row * 128 + ((unit ^ (row & 7)) << 4);
            if constexpr (PL == 1) {
                *reinterpret_cast<uint4*>(to) =
                    pairs ? make_uint4(raw[i][0], raw[i][1], raw[i][2], raw[i][3])
                          : make_uint4(raw[i][0] | raw[i][1] << 16, raw[i][2] | raw[i][3] << 16, raw[i][4] | raw[i][5] << 16, raw[i][6] | raw[i][7] << 16);
            } else {
                uint32_t part[4][3];
#pragma unroll
                for (int k = 0; k < 4; ++k) split_pair(__uint_as_float(raw[i][2 * k]), __uint_as_float(raw[i][2 * k + 1]), part[k]);
#pragma unroll
                for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(to + k * plane) = make_uint4(part[0][k], part[1][k], part[2][k], part[3][k]);
            }
        }
    }
}

// Where the run counts of 32 rows each are kept: behind the turns.
__device__ __forceinline__ int* low_adapter_runs(uint32_t* turns) { return reinterpret_cast<int*>(turns + 8); }

// bfloat16 part `part` of 16 float32 values (by truncation, each rest exact).
__device__ __forceinline__ void part_of_16(float (&f)[16], int part, uint4 (&v)[2]) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t k[3];
        split_pair(f[2 * i], f[2 * i + 1], k);
        r[i] = part == 0 ? k[0] : part == 1 ? k[1] : k[2];
    }
    v[0] = make_uint4(r[0], r[1], r[2], r[3]);
    v[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// 16 ranks of an adapter's b in column m, from q on, and of a row's u.
__device__ __forceinline__ void ranks_of_b(const ProductParams& p, int l, int64_t m, int q, uint32_t (&raw)[8]) {
    const int rank = static_cast<int>(p.rank), width = m < p.N ? rank - q : 0;
    const uint16_t* b = static_cast<const uint16_t*>(p.b) + (width > 0 ? (int64_t(l) * p.N + m) * rank + q : 0);
    if (rank % 8 == 0 && (reinterpret_cast<uintptr_t>(p.b) & 15) == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 x = k * 8 < width ? __ldg(reinterpret_cast<const uint4*>(b) + k) : make_uint4(0, 0, 0, 0);
            raw[4 * k] = x.x, raw[4 * k + 1] = x.y, raw[4 * k + 2] = x.z, raw[4 * k + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            raw[k] = 2 * k < width ? __ldg(b + 2 * k) : 0;
            if (2 * k + 1 < width) raw[k] |= static_cast<uint32_t>(__ldg(b + 2 * k + 1)) << 16;
        }
    }
}
// Two 16-bit values of b with 0 in the place of an infinity or NaN, whose exponent bits are all ones.
__device__ __forceinline__ uint32_t finite_pair(uint32_t two, uint32_t exponent) {
    return two & (((two & exponent) == exponent ? 0u : 0xffffu) | ((two >> 16 & exponent) == exponent ? 0u : 0xffff0000u));
}
__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// What finite_pair and its like kept out of the low-rank part of a tile, the
// terms with an infinity or NaN in b or u, to their places: a pass of its own
// over the accumulators after the tile's, and no part of the loop there, where
// its registers would cost the calls that have no such terms.  The warp's
// columns c0, c0 + STEP, .. W at a time, of lane column m; the sums go to
// `part`, a part of a split tile, or to the result.
template <int W, int STEP>
__device__ __noinline__ void add_strange(const KernelArgs& a, uint32_t from, const int* tile_adapter, int row0, int columns, int c0, int64_t m,
                                         bool in, float* part) {
    const ProductParams& p = a.p;
    const int rank = static_cast<int>(p.rank);
    __syncwarp();
    for (; c0 < columns; c0 += STEP) {
        float d[W];
        tmem_load(from + c0, d);
        tmem_wait(d);
#pragma unroll 1
        for (int j = 0; j < W && c0 + j < columns; ++j) {
            const int l = tile_adapter[c0 + j];
            if (l < 0 || !in) continue;
            const float* u = p.u + (int64_t(row0) + c0 + j) * rank;
            const uint16_t* b = static_cast<const uint16_t*>(p.b) + (int64_t(l) * p.N + m) * rank;
            float s = 0.0f, x = 0.0f;
            for (int k = 0; k < rank; ++k) {
                const float f = p.type == PT_BF16 ? __uint_as_float(static_cast<uint32_t>(b[k]) << 16) : __half2float(__ushort_as_half(b[k]));
                if (!is_finite(u[k]) || !is_finite(f)) s = fmaf(u[k], f, s);
            }
            if (s == 0.0f) continue;
#pragma unroll
            for (int k = 0; k < W; ++k) x = k == j ? d[k] : x;
            if (part) part[(c0 + j) * MT] = x + s;
            else if (p.out_type == PT_F32) static_cast<float*>(p.out)[(int64_t(row0) + c0 + j) * p.ldo + m] += s;     // with the pieces before
            else static_cast<uint16_t*>(p.out)[(int64_t(row0) + c0 + j) * p.ldo + m] = static_cast<uint16_t>(narrow_pair(x + s, 0.0f, p.out_type));
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void ranks_of_u(const ProductParams& p, bool in, int64_t row, int q, float (&f)[16]) {
    const int rank = static_cast<int>(p.rank), width = in ? rank - q : 0;
    const float* u = p.u + (width > 0 ? row * rank + q : 0);
#pragma unroll
    for (int k = 0; k < 16; ++k) f[k] = 0.0f;
    if (rank % 4 == 0) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 x = k < width ? *reinterpret_cast<const float4*>(u + k) : make_float4(0, 0, 0, 0);
            f[k] = x.x, f[k + 1] = x.y, f[k + 2] = x.z, f[k + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (k < width) f[k] = u[k];
    }
}

// One block of an adapter's part of the sum, for the rows [row, end) of the
// tile: up to four steps of 16 ranks, each one product of a part of b (A: a
// thread per lane of the tile) and a part of u (B: a thread per row, zeros
// outside the run).  The steps of 16 ranks follow one another: bfloat16 b:
// parts (b, u) = (0, 0), (0, 1), (0, 2); float16 b has two parts: and (1, 0),
// (1, 1); what is left out is below 2^-21.  A block's steps touch two groups
// of 16 ranks at most, which are loaded together.
// Every column of the tile meets this b, those outside the run with zeros, and
// 0 times an infinity or NaN is NaN: such values of b (and of u, whose parts
// would lose an infinity's sign) count as 0 here, and the drain warps add their
// terms to the run's own rows.  Returns whether this thread found one.
__device__ __forceinline__ bool lay_adapter(const ProductParams& p, int s0, int total, int pairs, int l, int64_t m, int row0, int base,
                                            int share, int row, int end, unsigned char* sa, unsigned char* sb, int tl) {
    const int j0 = s0 / pairs;
    bool strange = false;
    {
        uint32_t raw[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) ranks_of_b(p, l, m, (j0 + k) * 16, raw[k]);
        // the largest magnitude of each half tells
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) most = __vmaxu2(most, raw[k / 8][k % 8] & 0x7fff7fffu);
        const uint32_t exponent = p.type == PT_F16 ? 0x7c00u : 0x7f80u;
        if ((most & 0xffffu) >= exponent || most >> 16 >= exponent) {
            strange = true;
#pragma unroll
            for (int k = 0; k < 16; ++k) raw[k / 8][k % 8] = finite_pair(raw[k / 8][k % 8], exponent);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + i, second = s >= (j0 + 1) * pairs ? 1 : 0, pair = s - (j0 + second) * pairs;
            if (s >= total) break;
            uint32_t r[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = second ? raw[1][k] : raw[0][k];
            uint4 v[2] = {make_uint4(r[0], r[1], r[2], r[3]), make_uint4(r[4], r[5], r[6], r[7])};
            if (p.type == PT_F16) {
                float f[16];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r[k]));
                    f[2 * k] = x.x, f[2 * k + 1] = x.y;
                }
                part_of_16(f, pair >= 3 ? 1 : 0, v);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4*>(sa + tl * 128 + (((2 * i + k) ^ (tl & 7)) << 4)) = v[k];
        }
    }
    for (int r = tl; r < share; r += 128) {
        const bool in = base + r >= row && base + r < end;
        float f[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k) ranks_of_u(p, in, int64_t(row0) + base + r, (j0 + k) * 16, f[k]);
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) most = max(most, __float_as_uint(f[k / 16][k % 16]) & 0x7fffffffu);
        if (most >= 0x7f800000u) {
            strange = true;
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (!is_finite(f[k / 16][k % 16])) f[k / 16][k % 16] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + i, second = s >= (j0 + 1) * pairs ? 1 : 0, pair = s - (j0 + second) * pairs;
            if (s >= total) break;
            float g[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) g[k] = second ? f[1][k] : f[0][k];
            uint4 v[2];
            part_of_16(g, pair >= 3 ? pair - 3 : pair, v);
#pragma unroll
            for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4*>(sb + r * 128 + (((2 * i + k) ^ (r & 7)) << 4)) = v[k];
        }
    }
    return strange;
}

// Whether the stage of a block already holds its A operand: with two stages
// and a sum of one or two blocks, every tile of a segment and the one before
// use the same.  STREAMS: 1 for a role that sees every second block, which is
// always in one stage, 2 for one that sees all.
template <int MODE, bool ON, int STREAMS>
struct Kept {
    int seg[STREAMS], m0[STREAMS], kb[STREAMS];
    __device__ __forceinline__ Kept() {
#pragma unroll
        for (int i = 0; i < STREAMS; ++i) seg[i] = -1;
    }
    __device__ __forceinline__ bool a(const Item& t, int block) {
        if (!ON || MODE == PRODUCT_WEIGHTS) return false;
        const bool same = seg[0] == t.seg && m0[0] == t.m0 && kb[0] == block;
#pragma unroll
        for (int i = 0; i + 1 < STREAMS; ++i) seg[i] = seg[i + 1], m0[i] = m0[i + 1], kb[i] = kb[i + 1];
        seg[STREAMS - 1] = t.seg, m0[STREAMS - 1] = t.m0, kb[STREAMS - 1] = block;
        return same;
    }
};

// ---------------------------------------------------------------------------

template <int MODE, bool TENSOR, int NT, int PL, int CG>
__global__ void __launch_bounds__(threads_of<MODE, TENSOR, PL>(), 1)
product_kernel(const __grid_constant__ KernelArgs a, const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b) {
    using R = Ring<MODE, NT, PL, CG, TENSOR>;
    static_assert(CG == 1 || (TENSOR && PL == 1), "pairs take their operands as they are copied");
    constexpr bool GATED = MODE == PRODUCT_GATED;
    static_assert(!GATED || TENSOR, "operands that tensor copies cannot take are gated by a kernel of their own");
    constexpr int LANES = GATED ? MT / 2 : MT;
    constexpr int HALVES = PL == 1 ? 1 : 2;          // copies of 128 bytes that make 64 values
    extern __shared__ unsigned char raw[];
    unsigned char* stages = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char* staging = stages + R::ALL_STAGES * R::STAGE;      // 16-byte aligned, as all that follows it
    int* near = reinterpret_cast<int*>(staging + R::STAGED);
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + R::STAGED + R::NEAR);   // CG == 2: CTA 0's count
    uint64_t* empty = full + R::STAGES;
    uint64_t* landed = empty + R::STAGES;          // a stage whose tail has to be zeroed has arrived
    uint64_t* acc_full = landed + R::STAGES;
    uint64_t* acc_empty = acc_full + 2;            // CG == 2: CTA 0's count
    uint64_t* drain = acc_empty + 2;
    uint64_t* low_full = drain + 1;                // CG == 2: CTA 0's count
    uint64_t* low_empty = low_full + 1;
    uint64_t* low_done = low_empty + 1;            // the low-rank warps of both CTAs are through with a tile
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(low_done + LOW_TILES);
    int* low_steps = reinterpret_cast<int*>(tmem_at + 1);                // steps of 16 in the low-rank stage; + 8: the tile's last
    uint32_t* low_turns = reinterpret_cast<uint32_t*>(low_steps + 1);          // [8]: rows with another adapter than the one before
    uint32_t* low_strange = tmem_at + 20;                        // infinities or NaN were kept out of a low-rank part
    int* tile_adapter = reinterpret_cast<int*>(tmem_at + 32);    // [NT], the drain warps'
    int* low_adapter = tile_adapter + NT;                        // [NT], the low-rank warps'
    if (PL > 1 && !GATED) staging = reinterpret_cast<unsigned char*>(near);
    // a part of a split tile's sum [columns][128 lanes], where the stages were once its MMAs are done
    float* cluster_part = reinterpret_cast<float*>(stages);
    static_assert(R::STAGES * R::STAGE >= NT * MT * 4, "room for a part");
    const ProductParams& p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool split = a.parts > 1;                // the parts of a tile are a cluster
    const uint32_t in_cluster = CG == 2 || split ? cluster_rank() : 0;
    const int rank = CG == 2 ? static_cast<int>(in_cluster & 1) : 0;
    const uint32_t lead = in_cluster & ~1u;
    uint32_t first = blockIdx.x / CG, stride = gridDim.x / CG;

    const bool is_near = p.S <= NEAR_SEGMENTS;
    const int* beg = is_near ? near : a.far;
    const int* pre = is_near ? near + NEAR_SEGMENTS + 1 : a.far + p.S + 1;
    if (warp == 0) tmem_alloc<CG>(tmem_at, 2 * R::ACC);
    if (tid == 0) {
        for (int i = 0; i < R::STAGES; ++i) {
            mbar_init(full + i, TENSOR && PL == 1 ? CG : LOADERS / 32);
            mbar_init(empty + i, 1);
            mbar_init(landed + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, EPW * CG);
        }
        mbar_init(drain, 1);
        mbar_init(low_full, 4 * CG);
        mbar_init(low_empty, 1);
        for (int i = 0; i < LOW_TILES; ++i) mbar_init(low_done + i, 4 * CG);
        if (R::LOW) *low_strange = 0;
        fence_mbarrier_init();
        if (TENSOR) {
            tensor_prefetch(&map_a);
            tensor_prefetch(&map_b);
        }
    }
    if (is_near && MODE != PRODUCT_ADAPTERS && p.S > 0) fill_prefix<MODE, NT, 1>(a, near, near + NEAR_SEGMENTS + 1);
    // (PL == 3: that space is the staging)
    const int* near_offsets = MODE == PRODUCT_ADAPTERS && PL == 1 && is_near ? near : nullptr;
    if (near_offsets && p.S > 0)
        for (int64_t s = tid; s <= p.S; s += blockDim.x) {
            near[s] = offset_at(p, s);
            if (s < p.S) near[NEAR_SEGMENTS + 1 + s] = __ldg(p.index + s);
        }
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || split) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    uint32_t items;
    // (the caps: offsets that decrease name more items than there can be)
    if (MODE == PRODUCT_WEIGHTS) items = static_cast<uint32_t>(min(int64_t(pre[p.S]), p.S + p.R / a.chunk) * (a.mtiles * a.ntiles));
    else if (MODE == PRODUCT_ADAPTERS) items = static_cast<uint32_t>(a.row_tiles * a.mtiles * a.parts);
    else items = static_cast<uint32_t>((p.S > 0 ? min(int64_t(pre[p.S]), a.row_tiles) : 0) * a.mtiles * a.parts);
    constexpr bool KEEPS = (MODE == PRODUCT_FORWARD || GATED) && PL == 3 && R::STAGES == 2;      // see Kept
    if ((MODE != PRODUCT_ADAPTERS && !is_near) || (KEEPS && a.kblocks <= 2 && a.mtiles == 1 && !split)) {
        // many segments, whose prefix is in memory: neighbouring items, so that
        // the next one's segment is found by a step or two instead of a search;
        // or the next one can keep this one's matrix (mm of 1,000,000 x 64 rows
        // in 50 segments: 117 -> 106 us)
        const uint32_t each = (items + stride - 1) / stride;
        first *= each;
        items = min(items, first + each);
        stride = 1;
    }
    const bool a_outer = MODE == PRODUCT_WEIGHTS || !p.trans;    // the operand's contiguous dimension is m, not the sum
    constexpr bool b_outer = MODE == PRODUCT_WEIGHTS;

    // Extents of a tile: lanes of this CTA that exist, columns, and columns per CTA.
    auto lanes_of = [&](const Item& t) {
        const int64_t left = a.cols_m - t.m0 - rank * LANES;
        return static_cast<int>(left < LANES ? (left < 0 ? 0 : left) : LANES);
    };
    auto columns_of = [&](const Item& t) {
        return MODE == PRODUCT_WEIGHTS ? static_cast<int>(a.cols_n - t.n0 < NT ? a.cols_n - t.n0 : NT) : t.rows;
    };
    auto share_of = [&](int columns) { return ((columns + CG - 1) / CG + 15) & ~15; };
    // The last block of a weights' sum reaches past the segment: those rows are zeroed once they have arrived.
    auto has_tail = [&](const Item& t, int kb) { return PL == 1 && MODE == PRODUCT_WEIGHTS && kb + 1 == t.kb1 && (t.rows & 15) != 0; };

    constexpr bool TWIN = MODE == PRODUCT_FORWARD && TENSOR && PL == 3;
    const bool twin = TWIN && a.twin;

    if (TENSOR && (warp == 1 || warp == 3)) {
        // ---- producers: two, which take turns at the blocks (one thread's
        // chain of wait, expect and copies for a block took longer than its MMAs) ----
        const uint32_t turn = warp >> 1;
        if (elect_one()) {
            uint32_t next = turn, base = 0;                // this producer's next block; the item's first
            uint32_t st = turn % R::STAGES, ph = turn < R::STAGES ? 1 : 0;
            bool ok = true;
            Kept<MODE, R::STAGES == 2 && PL == 3, 1> keeps;
            Item t;
            for (uint32_t i = first; ok && i < items; i += stride) {
                item_at<MODE, NT, CG>(a, beg, pre, i, t);
                const uint32_t blocks = t.kb1 > t.kb0 ? t.kb1 - t.kb0 : 0;
                const int columns = columns_of(t), share = share_of(columns), lanes = lanes_of(t);
                const int a_boxes = GATED ? (lanes > 0 ? 2 : 0) : a_outer ? (lanes + 63) / 64 : (lanes + MT - 1) / MT;
                const int b_boxes = b_outer ? (share + 63) / 64 : (share + a.box_rows - 1) / a.box_rows;
                const uint32_t a_bytes = a_boxes * (a_outer ? 8192 : a.a_rows * 128) * HALVES * (twin ? 2 : 1), b_bytes = b_boxes * (b_outer ? 8192 : a.box_rows * 128) * HALVES;
                const int m0 = t.m0 + rank * LANES;
                uint32_t other_bytes = 0;
                if (CG == 2) {
                    const int64_t left = a.cols_m - t.m0 - LANES;
                    const int other = static_cast<int>(left < LANES ? (left < 0 ? 0 : left) : LANES);
                    other_bytes = b_bytes + (GATED ? (other > 0 ? 2 : 0) * (a_outer ? 8192 : a.a_rows * 128)
                                                   : a_outer ? (other + 63) / 64 * 8192 : (other + MT - 1) / MT * a.a_rows * 128);
                }
                int64_t m = t.seg;
                if (MODE == PRODUCT_FORWARD && p.index) m = __ldg(p.index + t.seg);
                for (; next - base < blocks; next += 2) {
                    const int kb = t.kb0 + static_cast<int>(next - base);
                    ok = wait_for<CG>(empty + st, ph, p.status);
                    if (!ok) break;
                    unsigned char* sa = stages + st * R::STAGE;
                    unsigned char* sb = sa + PL * R::A_PLANE;
                    const bool tail = has_tail(t, kb);
                    const uint32_t bar = tail || PL > 1 ? smem_u32(landed + st) : lead_addr<CG>(full + st, lead);
                    const bool keep = keeps.a(t, kb);
                    if (tail || PL > 1) {
                        mbar_arrive_expect_tx(landed + st, (keep ? 0 : a_bytes) + b_bytes);
                    } else if (rank == 0) {      // both arrivals, and the bytes of both CTAs
                        mbar_arrive_expect_tx(full + st, a_bytes + b_bytes + other_bytes);
                        if (CG == 2) mbar_arrive(full + st);
                    }
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        unsigned char* da = sa + (PL == 1 ? 0 : (1 + h) * R::A_PLANE);
                        unsigned char* db = sb + (PL == 1 ? 0 : (1 + h) * R::B_PLANE);
                        if (MODE == PRODUCT_WEIGHTS) {
                            const int r = t.row0 + kb * KB, n0 = t.n0 + rank * share + h * 32;
                            for (int x = 0; x < a_boxes; ++x) tensor_load_2d<CG>(da + x * 8192, &map_a, m0 + x * 64 + h * 32, r, bar);
                            for (int x = 0; x < b_boxes; ++x) tensor_load_2d<CG>(db + x * 8192, &map_b, n0 + x * 64, r, bar);
                        } else {
                            const int r0 = t.row0 + rank * share, k0 = kb * KB;
                            if (keep) {
                            } else if (GATED) {
                                // the two projections' 64 columns, one after the other
                                for (int x = 0; x < a_boxes; ++x) {
                                    if (a_outer) tensor_load_4d<CG>(da + x * 8192, &map_a, m0 + h * 32, x, k0, static_cast<int>(m), bar);
                                    else tensor_load_4d<CG>(da + x * 8192, &map_a, k0 + h * 32, m0, x, static_cast<int>(m), bar);
                                }
                            } else if (twin) {
                                for (int x = 0; x < 2; ++x)
                                    tensor_load_3d<CG>(da + x * 8192, &map_a, a_outer ? m0 + h * 32 : k0 + h * 32, a_outer ? k0 : m0, static_cast<int>(m), bar);
                            } else if (a_outer) {
                                for (int x = 0; x < a_boxes; ++x)
                                    tensor_load_3d<CG>(da + x * 8192, &map_a, m0 + x * 64 + h * 32, k0, static_cast<int>(m), bar);
                            } else if (a_boxes > 0) {
                                tensor_load_3d<CG>(da, &map_a, k0 + h * 32, m0, static_cast<int>(m), bar);
                            }
                            for (int x = 0; x < b_boxes; ++x)
                                tensor_load_2d<CG>(db + x * a.box_rows * 128, &map_b, k0 + h * 32, r0 + x * a.box_rows, bar);
                        }
                    }
                    if ((st += 2) >= R::STAGES) {
                        st -= R::STAGES;
                        ph ^= 1;
                    }
                }
                base += blocks;
            }
            if (rank == 0 && !ok) {
                // something gave up: the copies in flight still land before this CTA's shared memory goes away
                for (uint32_t j = next > R::STAGES ? next - R::STAGES : 0; j < next; ++j)
                    wait_for<CG>((PL > 1 ? landed : full) + j % R::STAGES, (j / R::STAGES) & 1, p.status);
            }
        }
        __syncwarp();
    } else if ((!TENSOR || PL > 1) && warp >= LOAD_WARP) {
        // ---- loaders: split what the producers copied, or load by themselves ----
        uint32_t st = 0, ph = 0;
        bool ok = true;
        Kept<MODE, R::STAGES == 2 && PL == 3, 2> keeps;
        Item t;
        for (uint32_t i = first; ok && i < items; i += stride) {
            item_at<MODE, NT, CG>(a, beg, pre, i, t);
            const int share = share_of(columns_of(t)), lanes = lanes_of(t);
            const int a_rows = twin || GATED ? (a_outer ? MT : 64 + a.a_rows) : a_outer ? (lanes + 63) & ~63 : a.a_rows, b_rows = b_outer ? (share + 63) & ~63 : share;
            int64_t m = t.seg;
            if (MODE == PRODUCT_FORWARD && p.index) m = __ldg(p.index + t.seg);
            for (int kb = t.kb0; kb < t.kb1; ++kb) {
                // (an empty stage's barrier is a phase behind a copied one's)
                ok = warp_wait<CG>((TENSOR ? landed : empty) + st, TENSOR ? ph : ph ^ 1, p.status);
                if (!ok) break;
                unsigned char* sa = stages + st * R::STAGE;
                unsigned char* sb = sa + PL * R::A_PLANE;
                const bool keep = keeps.a(t, kb);
                const int64_t left = (MODE == PRODUCT_WEIGHTS ? t.rows : p.K) - int64_t(kb) * KB;
                const int used = left < KB ? static_cast<int>(left + 15) & ~15 : KB;
                if constexpr (TENSOR) {
                    // rows past the segment's end belong to others: they count as zeros
                    const int valid = MODE == PRODUCT_WEIGHTS ? t.rows - kb * KB : KB;
                    if (!keep) split_rows(a_rows, valid, sa, R::A_PLANE);
                    split_rows(b_rows, valid, sb, R::B_PLANE);
                } else {
                    const void* w = static_cast<const unsigned char*>(p.w) + m * p.stride_w * (PL == 1 ? 2 : 4);
                    const int64_t k = int64_t(kb) * KB;
                    if (keep) {
                    } else if (a_outer) {
                        load_any<PL>(Operand{w, p.ldw, k, p.K, t.m0, a.cols_m, a_rows, true, used}, sa, R::A_PLANE);
                    } else {
                        load_any<PL>(Operand{w, p.ldw, t.m0, a.cols_m, k, p.K, a_rows, false, used}, sa, R::A_PLANE);
                    }
                    load_any<PL>(Operand{p.x, p.ldx, t.row0, t.row0 + t.rows, k, p.K, b_rows, false, used}, sb, R::B_PLANE);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) lead_arrive<CG>(full + st, lead, true);
                if (++st == R::STAGES) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (TENSOR && PL == 1 && MODE == PRODUCT_WEIGHTS && warp == 2) {
        // ---- tails ----
        uint32_t st = 0, seen = 0;        // a parity per stage
        bool ok = true;
        Item t;
        for (uint32_t i = first; ok && i < items; i += stride) {
            item_at<MODE, NT, CG>(a, beg, pre, i, t);
            if (t.kb1 <= t.kb0) continue;
            st = (st + (t.kb1 - t.kb0 - 1)) % R::STAGES;
            if (has_tail(t, t.kb1 - 1)) {
                ok = warp_wait<CG>(landed + st, seen >> st & 1, p.status);
                if (!ok) break;
                seen ^= 1u << st;
                // rows past the segment's end belong to others: zero them up to the last step's end
                const int boxes_a = (lanes_of(t) + 63) / 64, boxes = boxes_a + (share_of(columns_of(t)) + 63) / 64;
                const int tail = t.rows & (KB - 1), zero = (16 - (t.rows & 15)) * 8;
                for (int u = lane; u < zero * boxes; u += 32) {
                    const int x = u / zero, q = u - x * zero;
                    unsigned char* box = stages + st * R::STAGE + (x < boxes_a ? x * 8192 : PL * R::A_PLANE + (x - boxes_a) * 8192);
                    *reinterpret_cast<uint4*>(box + tail * 128 + q * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) lead_arrive<CG>(full + st, lead, true);
            }
            if (++st == R::STAGES) st = 0;
        }
    } else if (R::LOW && warp >= LOW_WARP) {
        // ---- the adapters' part of tiles with few runs of rows, as further blocks of the sum ----
        if (p.u) {
            grid_wait();
            const int tl = tid - LOW_WARP * 32;
            unsigned char* sa = stages + R::STAGES * R::STAGE;
            unsigned char* sb = sa + R::A_PLANE;
            const int pairs = p.type == PT_BF16 ? 3 : 5, total = static_cast<int>((p.rank + 15) / 16) * pairs;
            uint32_t ph = 1, tiles = 0;
            bool ok = true;
            Item t;
            for (uint32_t i = first; ok && i < items; i += stride) {
                item_at<MODE, NT, CG>(a, beg, pre, i, t);
                if (t.kb1 <= t.kb0 || t.part != 0) continue;
                bool found = false;                    // an infinity or NaN in the tile's low-rank part
                for (int r = tl; r < t.rows; r += 128) low_adapter[r] = adapter_of(p, near_offsets, t.row0 + r);
                bar_low();
                int runs = 0;
                for (int r = tl; r - tl < NT; r += 128) {
                    const int l = r < t.rows ? low_adapter[r] : -2, before = r > 0 && r < t.rows ? low_adapter[r - 1] : -2;
                    const uint32_t turns = __ballot_sync(0xffffffffu, r < t.rows && l != before);
                    const uint32_t starts = __ballot_sync(0xffffffffu, r < t.rows && l >= 0 && l != before);
                    if (lane == 0) low_turns[r >> 5] = turns, low_adapter_runs(low_turns)[r >> 5] = __popc(starts);
                }
                bar_low();
                for (int k = 0; k < NT / 32; ++k) runs += low_adapter_runs(low_turns)[k];
                const bool mine = runs > 0 && runs * LOW_RUN <= t.rows;
                int row = 0;                           // the next run's first row
                bool last = false;
                do {
                    int end = 0, l = -1;
                    if (mine) {
                        // the next run with an adapter
                        do {
                            l = low_adapter[row];
                            end = t.rows;
                            for (int k = (row + 1) >> 5; k < NT / 32; ++k) {
                                const uint32_t m = low_turns[k] & (k == (row + 1) >> 5 ? ~0u << ((row + 1) & 31) : ~0u);
                                if (m) {
                                    end = min(t.rows, k * 32 + __ffs(m) - 1);
                                    break;
                                }
                            }
                            if (l < 0) row = end;
                        } while (l < 0);
                        --runs;
                    }
                    for (int s0 = 0; ok && s0 < (mine ? total : 1); s0 += 4) {
                        ok = bar_low_all(wait_for<CG>(low_empty, ph, p.status));
                        if (!ok) break;
                        ph ^= 1;
                        last = runs == 0 && s0 + 4 >= total;
                        if (!mine) last = true;
                        if (mine) {
                            found |= lay_adapter(p, s0, total, pairs, l, t.m0 + rank * MT + tl, t.row0, rank * share_of(t.rows), share_of(t.rows),
                                                 row, end, sa, sb, tl);
                        }
                        if (tl == 0) *low_steps = (mine ? min(4, total - s0) : 0) | (last ? 8 : 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) lead_arrive<CG>(low_full, lead, true);
                    }
                    row = end;
                } while (ok && !last);
                found = __any_sync(0xffffffffu, found);
                if (lane == 0) {
                    // (u's rows are this CTA's share, and the drain warps of both need them)
                    if (found) *reinterpret_cast<volatile uint32_t*>(low_strange) = 1;
                    if (CG == 2 && found) cluster_store(cluster_addr(low_strange, in_cluster ^ 1), 1);
                    arrive_both<CG>(low_done + tiles % LOW_TILES, lead, found);
                }
                ++tiles;
                bar_low();        // the table has been read
            }
        }
        __syncwarp();
    } else if (warp == 0 && rank == 0) {
        // ---- MMA ----
        if (elect_one()) {
            uint32_t st = 0, ph = 0, buf = 0, bph = 1, low_ph = 0;
            bool ok = true;
            const uint32_t type = p.type == PT_F16 ? 0 : 1;
            // descriptors of the first stage; a step of 16 and a stage add to the address field
            const uint32_t a_step = (a_outer ? 2048 : 32) >> 4, b_step = (b_outer ? 2048 : 32) >> 4;
            const uint64_t a_desc = tc_smem_desc(smem_u32(stages), 8192);
            const uint64_t b_desc = tc_smem_desc(smem_u32(stages) + PL * R::A_PLANE, 8192);
            Item t;
            for (uint32_t i = first; ok && i < items; i += stride) {
                item_at<MODE, NT, CG>(a, beg, pre, i, t);
                const uint32_t idesc = tc_idesc(type, MT * CG, CG * share_of(columns_of(t)), a_outer, b_outer);
                [[maybe_unused]] const uint32_t wide_idesc = tc_idesc(type, MT, NT + share_of(columns_of(t)), a_outer, b_outer);
                const int64_t sum = MODE == PRODUCT_WEIGHTS ? t.rows : p.K;
                bool low_left = R::LOW && p.u && t.part == 0;
                for (int piece = t.kb0; ok && piece < t.kb1; piece += a.flush) {
                    const int piece_end = t.kb1 - piece < a.flush ? t.kb1 : piece + a.flush;
                    ok = wait_for<CG>(acc_empty + buf, bph, p.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + buf * R::ACC;
                    for (int kb = piece; kb < piece_end; ++kb) {
                        ok = wait_for<CG>(full + st, ph, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        const int64_t left = sum - int64_t(kb) * KB;
                        const uint64_t da = a_desc + st * (R::STAGE >> 4), db = b_desc + st * (R::STAGE >> 4);
#pragma unroll
                        for (int k = 0; k < KB / 16; ++k) {
                            if (k > 0 && k * 16 >= left) break;
                            const bool add = kb > piece || k > 0;
                            if constexpr (PL == 1) {
                                tc_mma<CG>(acc, da + k * a_step, db + k * b_step, idesc, add);
                            } else if constexpr (R::ROW3) {
                                // B's parts follow one another in shared memory: as one operand
                                // they take the first part of A all three, the second two and
                                // the third one, in three accumulators by size
#pragma unroll
                                for (int q = 0; q < 3; ++q)
                                    tc_mma<CG>(acc + q * NT, da + q * (R::A_PLANE >> 4) + k * a_step, db + k * b_step,
                                               tc_idesc(type, MT, (2 - q) * NT + share_of(columns_of(t)), a_outer, b_outer), add || q > 0);
                            } else {
                                // the products of parts: the largest alone, the others
                                // together; the first part of A takes two of B's at once
                                tc_mma<CG>(acc, da + k * a_step, db + k * b_step, wide_idesc, add);
                                constexpr int pa[4] = {2, 0, 1, 1}, pb[4] = {0, 2, 1, 0};
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    tc_mma<CG>(acc + NT, da + pa[q] * (R::A_PLANE >> 4) + k * a_step,
                                               db + pb[q] * (R::B_PLANE >> 4) + k * b_step, idesc, true);
                            }
                        }
                        tc_commit<CG>(empty + st, lead);
                        if (R::LOW && low_left && ((kb - t.kb0) % LOW_EVERY == LOW_EVERY - 1 || kb + 1 == t.kb1)) {
                            // the low-rank part's blocks, from a stage of their own, in
                            // between (a fixed order), so that they are laid out meanwhile;
                            // bfloat16 parts, whatever the type
                            const uint32_t low_idesc = tc_idesc(1, MT * CG, CG * share_of(columns_of(t)), false, false);
                            const uint64_t la = tc_smem_desc(smem_u32(stages + R::STAGES * R::STAGE), 8192);
                            const uint64_t lb = tc_smem_desc(smem_u32(stages + R::STAGES * R::STAGE) + R::A_PLANE, 8192);
                            do {
                                ok = wait_for<CG>(low_full, low_ph, p.status);
                                if (!ok) break;
                                low_ph ^= 1;
                                tc_fence_after();
                                const int steps = *reinterpret_cast<volatile int*>(low_steps);
                                low_left = (steps & 8) == 0;
                                for (int k = 0; k < (steps & 7); ++k) tc_mma<CG>(acc, la + 2 * k, lb + 2 * k, low_idesc, true);
                                tc_commit<CG>(low_empty, lead);
                            } while (low_left && kb + 1 == t.kb1);
                            if (!ok) break;
                        }
                        if (kb + 1 == piece_end) tc_commit<CG>(acc_full + buf, lead);
                        if (++st == R::STAGES) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                    if ((buf ^= 1) == 0) bph ^= 1;
                }
            }
            // no MMA is in flight when the memory goes away
            tc_commit<CG>(drain, lead, true);
            wait_for<CG>(drain, 0, p.status);
        }
        __syncwarp();
    } else if (warp >= EPI_WARP && warp < EPI_WARP + EPW) {
        // ---- drain ----
        const int quarter = (warp - EPI_WARP) & 3, group = (warp - EPI_WARP) / 4;   // which lanes; which columns
        const int td = tid - EPI_WARP * 32;
        constexpr int W = MODE == PRODUCT_ADAPTERS ? 8 : (TENSOR && PL == 1 ? 32 : 16), ROWS = W * (EPW / 4);    // columns at a time; of all warps
        constexpr bool BLOCKS = TENSOR && PL == 1 && MODE != PRODUCT_ADAPTERS;
        constexpr bool AHEAD = PL == 1;      // the next ones are loaded before these are stored, where registers allow
        unsigned char* const own_staging = staging + (warp - EPI_WARP) * R::STAGING;
        [[maybe_unused]] LowRank<PL, R::LOW> low(p, tile_adapter, own_staging, lane);
        if ((MODE == PRODUCT_FORWARD && !p.index) || GATED) {
            // rows in no segment
            const int b = p.S > 0 ? beg[0] : 0, e = p.S > 0 ? beg[p.S] : 0;
            const int64_t none = b + (p.R - (e > b ? e : b));
            const int64_t each = static_cast<int64_t>(gridDim.x) * (EPW * 32);
            for (int64_t i = blockIdx.x * (EPW * 32) + td; i < none * p.N; i += each) {
                const int64_t q = i / p.N, c = i - q * p.N, r = q < b ? q : (e > b ? e : b) + (q - b);
                if constexpr (GATED) {
                    if (p.pre && p.pre_type == PT_F32) static_cast<float*>(p.pre)[r * p.ldp + c] = 0.0f;
                    else if (p.pre) static_cast<uint16_t*>(p.pre)[r * p.ldp + c] = 0;
                    if (c >= a.cols_m) continue;
                }
                if (p.out_type == PT_F32) static_cast<float*>(p.out)[r * p.ldo + c] = 0.0f;
                else static_cast<uint16_t*>(p.out)[r * p.ldo + c] = 0;
            }
        }
        // the adapters' kernel starts beside the one that computes u, and
        // copies and multiplies meanwhile
        bool u_there = MODE != PRODUCT_ADAPTERS;
        uint32_t buf = 0, bph = 0;
        [[maybe_unused]] uint32_t low_tiles = 0;
        Item t;
        for (uint32_t i = first; i < items; i += stride) {
            item_at<MODE, NT, CG>(a, beg, pre, i, t);
            const bool summed = t.kb1 > t.kb0;
            const int n_left = columns_of(t);
            if constexpr (GATED) {
                // (warps that exchange values meet at barriers: all give up together)
                if (summed && !bar_drain_all(wait_for<CG>(acc_full + buf, bph, p.status))) break;
                tc_fence_after();
                const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * R::ACC;
                const int64_t m = t.m0 + rank * LANES + (quarter & 1) * 32;
                const int lanes = static_cast<int>(a.cols_m - m < 32 ? a.cols_m - m : 32);      // may be negative
                if (split) {
                    for (int c = group * W; c < n_left; c += ROWS) {
                        float v[W];
                        if (summed) load_sums<R, NT, PL, W>(from + c, v);
                        else
#pragma unroll
                            for (int j = 0; j < W; ++j) v[j] = 0.0f;
                        store_rows(cluster_part + quarter * 32 + c * MT + lane, MT, v, n_left - c, [](float x) { return x; });
                    }
                } else if (lanes > 0 && BLOCKS && a.wide_rows && (!p.pre || p.pre_type == PT_F32 || a.wide_pre)) {
                    gate_blocks<EPW / 4 * 32>(a, from, t.row0, group * 32, n_left, m, lanes, lane, quarter, group, own_staging, R::STAGING);
                } else if (lanes > 0) {
                    for (int c = group * W; c < n_left; c += ROWS) {
                        float v[W];
                        load_sums<R, NT, PL, W>(from + c, v);
                        gate_rows<PL != 1, W>(a, v, t.row0 + c, n_left - c, m, lanes, lane, quarter, group,
                                              own_staging + (PL > 1 ? (c / ROWS & 1) * (R::STAGING / 2) : 0), R::STAGING);
                    }
                }
                if (summed) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) lead_arrive<CG>(acc_empty + buf, lead, false);
                    if ((buf ^= 1) == 0) bph ^= 1;
                }
                continue;
            }
            const int64_t m = t.m0 + rank * MT + (twin ? quarter & 1 : quarter) * 32;           // the warp's first lane
            const int lanes = static_cast<int>(a.cols_m - m < 32 ? a.cols_m - m : 32);   // may be negative
            const int64_t slot = (t.slot * CG + rank) * NT * MT + quarter * 32;      // in floats
            bool scattered = true;      // the drain warps compute the tile's low-rank part
            if constexpr (MODE == PRODUCT_ADAPTERS) {
                bar_drain();       // the table of the tile before has been read
                for (int r = td; r < t.rows; r += EPW * 32) {
                    tile_adapter[r] = adapter_of(p, near_offsets, t.row0 + r);
                }
                bar_drain();
                if (R::LOW) {
                    int runs = 0;
                    for (int r = td; r - td < t.rows; r += EPW * 32) {
                        const bool starts = r < t.rows && tile_adapter[r] >= 0 && (r == 0 || tile_adapter[r - 1] != tile_adapter[r]);
                        runs += bar_drain_count(starts);
                    }
                    scattered = runs * LOW_RUN > t.rows;
                }
                if (!u_there) {
                    // u and the scratch are used from here on; b is asked for before
                    if (scattered && p.u && lane < lanes)
                        for (int c = group * W + t.part * ROWS; c < t.rows; c += ROWS * t.parts)
                            for (int j = 0; j < W && c + j < t.rows; ++j) {
                                const int l = tile_adapter[c + j];
                                if (l >= 0) prefetch_l2(static_cast<const unsigned char*>(p.b) + ((l * p.N + m + lane) * p.rank) * (PL == 1 ? 2 : 4));
                            }
                    grid_wait();
                    u_there = true;
                }
            }
            float factor = 1.0f;
            if (MODE == PRODUCT_FORWARD && p.scale) factor = __ldg(p.scale + __ldg(p.index + t.seg));
            // where the tile goes: its result, or (a part of a split sum) scratch
            const bool partial = t.parts > 1;
            const int64_t step = MODE == PRODUCT_WEIGHTS ? a.cols_m : p.ldo;
            const int64_t at = (MODE == PRODUCT_WEIGHTS ? (t.seg * a.cols_n + t.n0) * a.cols_m : t.row0 * p.ldo) + m;
            bool ok = true;
            int piece = t.kb0;
            do {
                const bool fresh = piece == t.kb0, final = t.kb1 - piece <= a.flush;
                const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * R::ACC;
                if constexpr (BLOCKS) {
                    if (!partial && a.wide_rows && p.out_type != PT_F32) {
                        if (summed) {
                            ok = warp_wait<CG>(acc_full + buf, bph, p.status);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        if (lanes > 0) store_tile<EPW / 4 * 32>(a, from, summed, group * 32, n_left, at, step, lanes, lane, own_staging);
                        if (summed) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) lead_arrive<CG>(acc_empty + buf, lead, false);
                            if ((buf ^= 1) == 0) bph ^= 1;
                        }
                        break;       // one piece: 16-bit results take the sums as they are
                    }
                }
                bool waiting = summed, strange = false;
                const int stride_c = twin ? 2 * ROWS : ROWS;
                int c = lanes > 0 ? (twin ? group + (quarter & 2) : group) * W : n_left;
                float d[W], lo[W];       // the accumulators' next columns
                auto load = [&](int at_c) {
                    tmem_load(from + at_c, d);
                    if constexpr (PL > 1) tmem_load(from + NT + at_c, lo);
                };
                if constexpr (MODE == PRODUCT_ADAPTERS)
                    if (final && scattered) low.begin(t.row0, t.rows, m + lane, c + t.part * ROWS);
                for (;;) {
                    float v[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) v[j] = 0.0f;
                    // the parts of a tile share its low-rank part
                    if constexpr (MODE == PRODUCT_ADAPTERS)
                        if (final && scattered && c < n_left && c / ROWS % t.parts == t.part) low.rows_of(v, c, c + ROWS * t.parts);
                    if (waiting) {
                        // (where the drain warps meet at barriers, they give up together)
                        const bool low_part = R::LOW && final && p.u && t.part == 0;
                        if (MODE == PRODUCT_ADAPTERS)
                            ok = bar_drain_all((!low_part || wait_for<CG>(low_done + low_tiles % LOW_TILES, low_tiles / LOW_TILES & 1, p.status)) && wait_for<CG>(acc_full + buf, bph, p.status));
                        else ok = warp_wait<CG>(acc_full + buf, bph, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        waiting = false;
                        // (once set, low_strange stays: a later tile then looks for terms that it may not have)
                        if (low_part) {
                            ++low_tiles;
                            strange = !scattered && *reinterpret_cast<volatile uint32_t*>(low_strange) != 0;
                        }
                        if (AHEAD && c < n_left) load(c);
                    }
                    if (c >= n_left) break;
                    const int n = n_left - c < W ? n_left - c : W;
                    if (summed) {
                        if constexpr (R::ROW3) {
                            // (the two small sums first)
                            tmem_load(from + NT + c, d);
                            tmem_load(from + 2 * NT + c, lo);
                            tmem_wait(d);
                            tmem_wait(lo);
#pragma unroll
                            for (int j = 0; j < W; ++j) lo[j] += d[j];
                            tmem_load(from + c, d);
                            tmem_wait(d);
                        } else {
                            if (!AHEAD) load(c);
                            tmem_wait(d);
                            if constexpr (PL > 1) tmem_wait(lo);
                        }
#pragma unroll
                        for (int j = 0; j < W; ++j) v[j] += PL > 1 ? d[j] + lo[j] : d[j];
                        if (AHEAD && c + stride_c < n_left) load(c + stride_c);
                        if (!fresh && (partial || lane < lanes)) {
                            // the sum so far, float32 wherever there is more than one piece
                            const float* so_far = partial ? a.partials + slot + int64_t(c) * MT : static_cast<const float*>(p.out) + at + c * step;
                            const int64_t s1 = partial ? MT : step;
#pragma unroll
                            for (int j = 0; j < W; ++j)
                                if (j < n) v[j] += so_far[j * s1 + lane];
                        }
                    }
                    if (partial) {
                        store_rows((MODE == PRODUCT_WEIGHTS ? a.partials + slot : cluster_part + quarter * 32) + int64_t(c) * MT + lane, MT, v, n,
                                   [](float x) { return x; });
                    } else {
                        if (MODE == PRODUCT_FORWARD && p.scale && final)
#pragma unroll
                            for (int j = 0; j < W; ++j) v[j] *= factor;
                        store_result(a, at + c * step, step, v, n, lanes, lane, own_staging);
                    }
                    c += stride_c;
                    if (c >= n_left) break;
                }
                if (!ok) break;
                if constexpr (R::LOW) {
                    if (strange && lanes > 0)
                        add_strange<W, ROWS>(a, from, tile_adapter, t.row0, n_left, group * W, m + lane, lane < lanes,
                                             partial ? cluster_part + quarter * 32 + lane : nullptr);
                }
                if (summed) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) lead_arrive<CG>(acc_empty + buf, lead, false);
                    if ((buf ^= 1) == 0) bph ^= 1;
                }
                piece = final ? t.kb1 : piece + a.flush;
            } while (piece < t.kb1);
            if (!ok) break;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (MODE != PRODUCT_WEIGHTS && split) {
        // The parts of a tile (a CTA, or a pair, has one) lie in the shared
        // memory of the cluster's CTAs; each CTA adds some of the rows, always
        // in the order of the parts.
        cluster_sync();
        if (first < items && warp >= EPI_WARP && warp < EPI_WARP + EPW) {
            constexpr int W = 8;
            const int quarter = (warp - EPI_WARP) & 3, group = (warp - EPI_WARP) / 4;
            Item t;
            item_at<MODE, NT, CG>(a, beg, pre, first, t);
            if constexpr (GATED) {
                // both projections of 32 columns of some rows
                const int64_t m = t.m0 + rank * LANES + (quarter & 1) * 32;
                const int lanes = static_cast<int>(a.cols_m - m < 32 ? a.cols_m - m : 32);
                for (int c = (t.part * EPW / 2 + group * 2 + (quarter >> 1)) * W; c < t.rows; c += t.parts * EPW / 2 * W) {
                    const int n = t.rows - c < W ? t.rows - c : W;
                    float v[2][W];
#pragma unroll
                    for (int j = 0; j < W; ++j) v[0][j] = v[1][j] = 0.0f;
#pragma unroll 4
                    for (int q = 0; q < t.parts; ++q) {
                        const uint32_t from = cluster_addr(cluster_part + c * MT + (quarter & 1) * 32 + lane, q * CG + rank);
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            if (j < n) v[0][j] += cluster_load(from + j * MT * 4), v[1][j] += cluster_load(from + (j * MT + LANES) * 4);
                    }
                    if (lane >= lanes) continue;
                    if (p.pre)
                        for (int h = 0; h < 2; ++h)
                            store_any(p.pre, p.pre_type, (int64_t(t.row0) + c) * p.ldp + h * a.cols_m + m + lane, p.ldp, v[h], n);
                    float f[W];
                    gate(p.activation, f, [&](int i) { return v[0][i]; }, [&](int i) { return v[1][i]; });
                    store_any(p.out, p.out_type, (int64_t(t.row0) + c) * p.ldo + m + lane, p.ldo, f, n);
                }
            } else {
            const int64_t m = t.m0 + rank * MT + quarter * 32;
            const int lanes = static_cast<int>(a.cols_m - m < 32 ? a.cols_m - m : 32);
            const float factor = MODE == PRODUCT_FORWARD && p.scale ? __ldg(p.scale + __ldg(p.index + t.seg)) : 1.0f;
            for (int c = (t.part * (EPW / 4) + group) * W; c < t.rows; c += t.parts * (EPW / 4) * W) {
                const int n = t.rows - c < W ? t.rows - c : W;
                float v[W];
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] = 0.0f;
#pragma unroll 4
                for (int q = 0; q < t.parts; ++q) {
                    const uint32_t from = cluster_addr(cluster_part + c * MT + quarter * 32 + lane, q * CG + rank);
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (j < n) v[j] += cluster_load(from + j * MT * 4);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] *= factor;
                store_result(a, (int64_t(t.row0) + c) * p.ldo + m, p.ldo, v, n, lanes, lane, staging + (warp - EPI_WARP) * R::STAGING);
            }
            }
        }
    }
    if (CG == 2 || split) cluster_sync();      // the others' MMAs, copies and sums use this CTA's memory
    if (warp == 0) {
        tc_fence_after();
        tmem_free<CG>(tmem, 2 * R::ACC);
    }
}

// Adds the parts of the split segments of the weights' product: a block per
// tile of a segment (blockIdx.x) and four of its columns at a time; warps w and
// w + 4 each add half of a column's parts, in order, and then the halves.
// Where there are more than twice as many segments as chunks of rows, a block
// stands for a chunk instead: one split segment at most starts in it, and no
// other segment after that one.  The search for it takes a few microseconds:
// 1.5 times as many, 100,000 x 64 float16, 20.0 us so and 18.5 by segments; 2.6
// times, 200,000 rows, 33.4 and 35.1.
constexpr int ADD_COLS = 4;

// The last segment that starts before `limit`, by all 256 threads of the block, or -1.
__device__ __forceinline__ int64_t last_before(const ProductParams& p, int64_t limit) {
    int64_t lo = 0, hi = p.S;
    do {
        const int64_t step = (hi - lo + 255) / 256, s = lo + threadIdx.x * step;
        const int count = __syncthreads_count(s < hi && offset_at(p, s) < limit);
        if (count == 0) return -1;
        lo += (count - 1) * step;
        hi = min(hi, lo + step);
    } while (hi - lo > 1);
    return lo;
}

template <int NT, int CG>
__global__ void __launch_bounds__(256) add_parts_kernel(const __grid_constant__ KernelArgs a) {
    __shared__ float4 half_sum[ADD_COLS][32];
    const ProductParams& p = a.p;
    const int per = a.mtiles * a.ntiles, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = blockIdx.x / per;
    const int r = static_cast<int>(blockIdx.x - item * per);
    const int64_t s = a.add_by_start ? last_before(p, (item + 1) * a.chunk) : item;
    if (s < 0) return;
    const int64_t b = offset_at(p, s), e = offset_at(p, s + 1);
    if (e - b <= a.chunk || (a.add_by_start && b / a.chunk != item)) return;
    const int parts = static_cast<int>((e - b + a.chunk - 1) / a.chunk), half = (parts + 1) / 2;
    const int rank = blockIdx.z;
    const int64_t m = (r % a.mtiles * CG + rank) * MT + lane * 4;
    const int n0 = r / a.mtiles * NT, columns = static_cast<int>(a.cols_n - n0 < NT ? a.cols_n - n0 : NT);
    const int q0 = warp < 4 ? 0 : half, q1 = warp < 4 ? half : parts;
    const int64_t j = b / a.chunk;
    for (int c0 = blockIdx.y * ADD_COLS; c0 < columns; c0 += gridDim.y * ADD_COLS) {
        const int c = c0 + (warp & 3);
        const bool in = m < a.cols_m && c < columns;
        float4 v = make_float4(0, 0, 0, 0);
        if (in) {
#pragma unroll 8
            for (int q = q0; q < q1; ++q) {
                const int64_t slot = (2 * (j + q) + (q == 0 ? 1 : 0)) * per + r;
                const float4 x = __ldcg(reinterpret_cast<const float4*>(a.partials + ((slot * CG + rank) * NT + c) * MT) + lane);
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
        }
        if (warp >= 4) half_sum[warp - 4][lane] = v;
        __syncthreads();
        if (warp < 4 && in) {
            const float4 x = half_sum[warp][lane];
            const float f[4] = {v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w};
            const int64_t at = (s * a.cols_n + n0 + c) * a.cols_m + m;
            for (int i = 0; i < 4; ++i) {
                if (m + i >= a.cols_m) break;
                if (p.out_type == PT_F32) static_cast<float*>(p.out)[at + i] = f[i];
                else if (p.out_type == PT_F16) static_cast<__half*>(p.out)[at + i] = __float2half_rn(f[i]);
                else static_cast<__nv_bfloat16*>(p.out)[at + i] = __float2bfloat16_rn(f[i]);
            }
        }
        __syncthreads();
    }
}

int64_t ceil_to(int64_t n, int64_t d) { return (n + d - 1) / d; }

// ---------------------------------------------------------------------------
// Rows of any alignment to rows of whole 16-byte units, one of those per thread
// at a time, several on their way.  What a tile's loader warps did with such rows
// was bound by the loads in flight that the L1 beside 200 KB of stages tracks,
// for every tile again.

// Division by a number that is known at the launch, by a product (Granlund and
// Montgomery, 1994), for dividends below 2^31.
struct Divisor {
    uint32_t d, mul, shift;
    explicit Divisor(uint32_t by = 1) : d(by), shift(0) {
        while ((uint64_t(1) << shift) < d) ++shift;
        mul = static_cast<uint32_t>((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d) / d + 1);
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct PackArgs {
    const void* src;
    unsigned char* dst;
    int64_t ld, stride, rows, cols, units;   // elements; rows of a matrix; columns of a packed row; 16-byte units of all
    int row_units;      // of a packed row
    int halves;         // 2: each row is two rows of `cols`, one after the other, that are packed as rows of their own
    int large;          // more units or rows than a Divisor divides
    Divisor by_row, by_mat;
};

// The 8 16-bit values from p on, all of them in the row: words where they lie on
// a word's border, else three words between two values.
__device__ __forceinline__ uint4 load_8(const uint16_t* p) {
    uint32_t w[4];
    if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {
        const uint32_t a = __ldg(p), e = __ldg(p + 7);
        uint32_t m[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) m[i] = __ldg(reinterpret_cast<const uint32_t*>(p + 1) + i);
        w[0] = a | m[0] << 16;
        w[1] = __funnelshift_l(m[0], m[1], 16);
        w[2] = __funnelshift_l(m[1], m[2], 16);
        w[3] = m[2] >> 16 | e << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// (64 x 520 rows of 666 float16, 44 MB there and back, each half a row of its own:
// a warp to a row and value by value 30 us, now 18 to 20.)
template <class T>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a) {
    constexpr int V = 16 / sizeof(T), AHEAD = 4;
    const int64_t step = int64_t(gridDim.x) * 256;
    for (int64_t u0 = int64_t(blockIdx.x) * 256 + threadIdx.x; u0 < a.units; u0 += AHEAD * step) {
        union {
            T v[V];
            uint4 u;
        } x[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t u = u0 + k * step;
            if (u >= a.units) break;
            int64_t row, mat;       // the packed row, its matrix
            if (a.large) row = u / a.row_units, mat = row / (a.rows * a.halves);
            else row = a.by_row.quotient(static_cast<uint32_t>(u)), mat = a.by_mat.quotient(static_cast<uint32_t>(row));
            const int64_t c = (u - row * a.row_units) * V, r = (a.halves == 2 ? row >> 1 : row) - mat * a.rows;
            const T* src = static_cast<const T*>(a.src) + mat * a.stride + r * a.ld + (a.halves == 2 && (row & 1) ? a.cols : 0) + c;
            bool whole = false;
            if constexpr (sizeof(T) == 2) {
                whole = c + V <= a.cols;
                if (whole) x[k].u = load_8(src);
            }
            if (!whole)
#pragma unroll
                for (int v = 0; v < V; ++v) x[k].v[v] = c + v < a.cols ? __ldg(src + v) : T(0);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (u0 + k * step < a.units) reinterpret_cast<uint4*>(a.dst)[u0 + k * step] = x[k].u;
    }
}

// Float32 rows of whole sums, rounded to the result.
template <class T>
__global__ void __launch_bounds__(256) round_kernel(const float* src, T* out, int64_t rows, int64_t cols, int64_t ldo) {
    const int64_t step = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * cols; i += step) {
        const int64_t r = i / cols;
        out[r * ldo + (i - r * cols)] = static_cast<T>(src[i]);
    }
}

// ---------------------------------------------------------------------------
// u[r, j] = scale * sum_k x[r, k] a[l, j, k] where requests have a row or a
// few: two warps per dot product, so that a's bytes (rank x K per request,
// bound by latency and L2) are spread over the whole GPU; a 128-lane tile per
// request would use 16 of its lanes and stream K through one SM.  96 rows of
// 96 requests, 4,096 columns, rank 16, the whole call: 25 us, with u by the
// tensor-core kernel 31; four ranks to a block, so that x is read a quarter as
// often.  The kernel is a chain of two loads and a reduction.  The shared
// product's kernel is launched beside it, but a CTA of that takes all registers
// of an SM and has to wait for this kernel's blocks there: of few blocks (one
// token: 4) its copies and products run beside these, of many (96 rows at rank
// 16: 384 on 152 SMs) only the launch does.

constexpr int DOT_RANKS = 4;      // ranks of a block, of one row; two warps each

template <class T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__global__ void __launch_bounds__(DOT_RANKS * 64, 3) lora_rows_kernel(const __grid_constant__ ProductParams p) {
    __shared__ int adapter;
    __shared__ float other[DOT_RANKS];
    grid_trigger();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31, slot = threadIdx.x >> 6, half = threadIdx.x >> 5 & 1;
    const int64_t j = int64_t(blockIdx.y) * DOT_RANKS + slot;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    // The row's first values are asked for before its adapter is known.
    constexpr int V = 16 / sizeof(T), AHEAD = 8, STEP = 64 * V;
    const bool whole_x = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && p.K % V == 0;
    const int64_t k0 = (half * 32 + lane) * V;
    uint4 xr[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        xr[i] = whole_x && k0 + i * STEP < p.K ? __ldg(reinterpret_cast<const uint4*>(x + k0 + i * STEP)) : make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) adapter = -1;
    __syncthreads();
    for (int64_t s = threadIdx.x; s < p.S; s += DOT_RANKS * 64) {
        const int l = __ldg(p.index + s);
        if (offset_at(p, s) <= row && row < offset_at(p, s + 1)) adapter = l;
    }
    __syncthreads();
    const int l = adapter;
    if (l < 0 || l >= p.L) return;
    float sum = 0.0f, sum2 = 0.0f;
    if (j < p.N) {
        const T* a = static_cast<const T*>(p.w) + (int64_t(l) * p.N + j) * p.K;
        if (whole_x && (reinterpret_cast<uintptr_t>(a) & 15) == 0) {
            for (int64_t k = k0; k < p.K; k += AHEAD * STEP) {
                uint4 ar[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    ar[i] = k + i * STEP < p.K ? __ldg(reinterpret_cast<const uint4*>(a + k + i * STEP)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const T *xv = reinterpret_cast<const T*>(&xr[i]), *av = reinterpret_cast<const T*>(&ar[i]);
                    // (a beyond the row's end counts as zero, whatever x holds there)
                    if (k + i * STEP < p.K)
#pragma unroll
                        for (int v = 0; v < V; v += 2) {
                            sum = fmaf(to_float(xv[v]), to_float(av[v]), sum);
                            sum2 = fmaf(to_float(xv[v + 1]), to_float(av[v + 1]), sum2);
                        }
                    const int64_t next = k + (AHEAD + i) * STEP;
                    if (next < p.K) xr[i] = __ldg(reinterpret_cast<const uint4*>(x + next));
                }
            }
        } else {
            for (int64_t k = half * 32 + lane; k < p.K; k += 64) sum = fmaf(to_float(__ldg(x + k)), to_float(__ldg(a + k)), sum);
        }
    }
    sum += sum2;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (half == 1 && lane == 0) other[slot] = sum;
    __syncthreads();
    if (half == 0 && lane == 0 && j < p.N)
        static_cast<float*>(p.out)[row * p.ldo + j] = (sum + other[slot]) * (p.scale ? __ldg(p.scale + l) : 1.0f);
}

// ---------------------------------------------------------------------------
// Tensor maps: 16-bit values, boxes of 64 columns, 128-byte swizzle.

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return EncodeFn(nullptr);
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// 128-byte rows of boxes: 64 16-bit or 32 float32 values.
bool make_map(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t ld, int64_t mats,
              int64_t stride, int box_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int rank = mats > 0 ? 3 : 2;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(mats)};
    const int size = type == PT_F32 ? 4 : 2;
    const cuuint64_t strides[2] = {cuuint64_t(ld) * size, cuuint64_t(stride) * size};
    const cuuint32_t box[3] = {cuuint32_t(128 / size), cuuint32_t(box_rows), 1}, each[3] = {1, 1, 1};
    return fn(map, type == PT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type == PT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void*>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Both projections' columns of the gated block's matrices, a box of 64 values x
// box_rows (the contiguous dimension's 64, or 32 float32, come first): [N, K] by
// projection and segment, or K rows of the two projections' N by segment.
bool make_gated_map(CUtensorMap* map, const ProductParams& p, int64_t half, int box_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t n = p.N / 2, k = p.K, size = p.type == PT_F32 ? 4 : 2;
    const cuuint64_t stride = p.S > 1 ? p.stride_w : (p.trans ? 2 * half : p.K * p.ldw);
    const cuuint32_t wide = 128 / static_cast<cuuint32_t>(size), rows = static_cast<cuuint32_t>(box_rows);
    const cuuint64_t dims_t[4] = {k, n, 2, cuuint64_t(p.S)}, dims[4] = {n, 2, k, cuuint64_t(p.S)};
    const cuuint64_t strides_t[3] = {p.ldw * size, half * size, stride * size}, strides[3] = {half * size, p.ldw * size, stride * size};
    const cuuint32_t box_t[4] = {wide, rows, 1, 1}, box[4] = {wide, 1, KB, 1}, each[4] = {1, 1, 1, 1};
    return fn(map, p.type == PT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : p.type == PT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(p.w), p.trans ? dims_t : dims, p.trans ? strides_t : strides, p.trans ? box_t : box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a tensor map can describe: 16-byte aligned, strides multiples of 16 bytes and below 2^40.
bool tensor_copyable(const void* base, int64_t stride, int type) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && stride % (type == PT_F32 ? 4 : 8) == 0 && stride < (int64_t(1) << 37);
}

template <int MODE, bool TENSOR, int NT, int PL, int CG>
cudaError_t launch_shape(const KernelArgs& a, const ProductPlan& plan, cudaStream_t stream) {
    // (a plan for other tiles would leave rows out)
    if (NT != product_tile_columns(a.p, plan)) return cudaErrorInvalidConfiguration;
    CUtensorMap ma{}, mb{};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (TENSOR) {
        // the driver call below needs the context, which a thread that has not
        // called the runtime yet (an autograd thread) does not have current
        e = cudaSetDevice(dev);
        if (e != cudaSuccess) return e;
        const ProductParams& p = a.p;
        bool ok;
        if (MODE == PRODUCT_WEIGHTS) {
            ok = make_map(&ma, p.type, p.w, p.N, p.R, p.ldw, 0, 0, KB) && make_map(&mb, p.type, p.x, p.K, p.R, p.ldx, 0, 0, KB);
        } else if (MODE == PRODUCT_GATED) {
            ok = make_gated_map(&ma, p, a.half_w, a.a_rows) && make_map(&mb, p.type, p.x, p.K, p.R, p.ldx, 0, 0, a.box_rows);
        } else {
            const int64_t mats = MODE == PRODUCT_ADAPTERS ? 1 : (p.index ? p.L : p.S);
            const int64_t rows = p.trans ? p.N : p.K, cols = p.trans ? p.K : p.N;
            ok = make_map(&ma, p.type, p.w, cols, rows, p.ldw, mats, mats > 1 ? p.stride_w : rows * p.ldw, p.trans ? a.a_rows : KB) &&
                 make_map(&mb, p.type, p.x, p.K, p.R, p.ldx, 0, 0, a.box_rows);
        }
        if (!ok) return cudaErrorInvalidValue;
    }
    if constexpr (MODE != PRODUCT_ADAPTERS) {
        if (a.p.S > NEAR_SEGMENTS) {
            prefix_kernel<MODE, NT><<<1, 1024, 0, stream>>>(a);
            e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
    }
    auto* kernel = product_kernel<MODE, TENSOR, NT, PL, CG>;
    using R = Ring<MODE, NT, PL, CG, TENSOR>;
    constexpr int smem = R::SMEM;
    cudaLaunchAttribute attr[2];
    int attrs = 0;
    if (CG > 1 || plan.parts > 1) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs].val.clusterDim.x = CG * plan.parts;
        attr[attrs].val.clusterDim.y = attr[attrs].val.clusterDim.z = 1;
        ++attrs;
    }
    // (not after a packing kernel: the producers read what it writes without waiting)
    const bool overlap = MODE == PRODUCT_ADAPTERS && a.p.overlap && !plan.pack_x && !plan.pack_w;
    if (overlap) {
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs].val.programmaticStreamSerializationAllowed = 1;
        ++attrs;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(plan.grid);
    cfg.blockDim = dim3(threads_of<MODE, TENSOR, PL>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 1 : 0;     // for the occupancy query
    static int resident[64] = {};       // most CTAs at a time, per device; callers hold the library's lock
    if (resident[dev] == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        int clusters = a.p.sms;
        if (CG > 1) {
            attr[0].val.clusterDim.x = CG;
            e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
            attr[0].val.clusterDim.x = CG * plan.parts;
            if (e != cudaSuccess) return e;
            if (clusters < 1) return cudaErrorInvalidConfiguration;
        }
        resident[dev] = clusters * CG;
    }
    cfg.numAttrs = attrs;
    // (a part has a CTA or a pair of its own)
    if (plan.parts == 1) cfg.gridDim = dim3(std::min(plan.grid, resident[dev]));
    e = cudaLaunchKernelEx(&cfg, kernel, a, ma, mb);
    if (e != cudaSuccess || plan.add_blocks == 0) return e;
    if constexpr (MODE == PRODUCT_WEIGHTS) {
        // (most blocks of chunks find no split segment, so there are few of them, which take several columns)
        const int64_t cols = ceil_to(std::min<int64_t>(a.cols_n, NT), ADD_COLS);
        add_parts_kernel<NT, CG><<<dim3(plan.add_blocks, static_cast<unsigned>(a.add_by_start ? std::min<int64_t>(cols, 8) : cols), CG), 256, 0, stream>>>(a);
        e = cudaGetLastError();
    }
    return e;
}

template <int MODE>
cudaError_t launch_mode(const KernelArgs& a, const ProductPlan& plan, cudaStream_t stream) {
    if (a.p.type == PT_F32 && plan.tensor)
        return plan.narrow ? launch_shape<MODE, true, 64, 3, 1>(a, plan, stream) : launch_shape<MODE, true, 128, 3, 1>(a, plan, stream);
    if constexpr (MODE == PRODUCT_FORWARD) {
        if (!plan.tensor) return a.p.type == PT_F32 ? launch_shape<MODE, false, 64, 3, 1>(a, plan, stream) : launch_shape<MODE, false, 64, 1, 1>(a, plan, stream);
    }
    if (plan.narrow) return launch_shape<MODE, true, 64, 1, 1>(a, plan, stream);
    return plan.pair ? launch_shape<MODE, true, 256, 1, 2>(a, plan, stream) : launch_shape<MODE, true, 256, 1, 1>(a, plan, stream);
}

}  // namespace

namespace {

// The second operand as matrices of contiguous rows.
struct MatShape {
    int64_t mats, rows, cols;
};
MatShape w_shape(int mode, const ProductParams& p) {
    if (mode == PRODUCT_WEIGHTS) return {1, p.R, p.N};
    if (mode == PRODUCT_ADAPTERS) return {1, p.N, p.K};
    return {p.index ? p.L : p.S, p.trans ? p.N : p.K, p.trans ? p.K : p.N};
}

// The gated block's two projections are copied apart: with contiguous columns each starts on a boundary of its own.
bool halves_apart(int mode, const ProductParams& p) { return mode == PRODUCT_GATED && !p.trans; }

int64_t packed_row(int64_t cols, int type) { return ceil_to(cols * (type == PT_F32 ? 4 : 2), 16) * 16; }   // bytes

}  // namespace

int product_tile_columns(const ProductParams& p, const ProductPlan& plan) { return plan.narrow ? 64 : (p.type == PT_F32 ? 128 : 256); }

ProductPlan plan_product(int mode, const ProductParams& p) {
    ProductPlan d{};
    const bool weights = mode == PRODUCT_WEIGHTS;
    const int64_t mats = mode == PRODUCT_FORWARD || mode == PRODUCT_GATED ? (p.index ? p.L : p.S) : 1;
    d.empty = p.K == 0 || p.R == 0 || mats == 0;
    const bool copy_x = tensor_copyable(p.x, p.ldx, p.type);
    const bool copy_w = tensor_copyable(p.w, p.ldw, p.type) && (mats == 1 || tensor_copyable(p.w, p.stride_w, p.type)) &&
                        (!halves_apart(mode, p) || p.N / 2 % (p.type == PT_F32 ? 4 : 8) == 0);
    const int64_t segments = mode == PRODUCT_ADAPTERS ? 1 : p.S;
    // An operand that tensor copies cannot take is laid out again first (one
    // more pass over it), except where most matrices are in no use: then the
    // loader warps take what is used as it is, at about a sixth of the speed.
    // (8,192 rows in 8 segments, 1,023 x 1,021 bfloat16: 40 us, by the loader
    // warps 174; 128 rows in 64 segments, 2,047 x 1,023: 152 us against 252.)
    if (!d.empty && !(copy_x && copy_w) && (weights || 2 * p.R >= mats)) {
        d.pack_x = !copy_x;
        d.pack_w = !copy_w;
    }
    d.tensor = !d.empty && (copy_x || d.pack_x) && (copy_w || d.pack_w);
    // few rows per segment, or too few tiles to go round: small tiles and a
    // deeper ring; weights: few columns of x.  The loader warps have small tiles alone.
    // The rows per segment are the mean, for lengths are on the device.  64
    // segments, bfloat16, small / large tiles: 2,048 x 1,024, 8 rows each 45.5 /
    // 47.3 us, 64 each 49.2 / 51.7, 16 with 3/4 of the rows in one segment 46.1 /
    // 48.0, 64 with 3/4 in one 60.4 / 51.5, all 4,096 in one 31.7 / 17.6; 1,024 x
    // 4,096: 81.3 / 85.1, 87.0 / 91.4, 89.1 / 85.7, 122 / 99.5, 56.2 / 27.0.
    d.narrow = !d.tensor || (weights ? p.K <= 64 : p.R <= 64 * segments || (p.N <= MT && p.R <= 128 * p.sms));
    const int NT = product_tile_columns(p, d);
    // two CTAs on a tile of twice the lanes, unless that leaves one of them without lanes
    // or so few tiles that their sums are split
    d.pair = d.tensor && p.type != PT_F32 && !d.narrow && (p.N > 1024 || ceil_to(p.N, MT) % 2 == 0);
    d.row_tiles = mode == PRODUCT_ADAPTERS ? ceil_to(p.R, NT) : std::min(segments, p.R) + p.R / NT;
    if (!weights && d.row_tiles * ceil_to(p.N, MT) * 2 <= p.sms * 27 / 32) d.pair = 0;
    const int cg = d.pair ? 2 : 1;
    d.mtiles = static_cast<int32_t>(ceil_to(p.N, MT * cg));
    d.ntiles = weights ? static_cast<int32_t>(ceil_to(p.K, NT)) : 1;
    d.parts = 1;
    d.part_blocks = static_cast<int32_t>(ceil_to(p.K, KB));
    d.chunk = std::max<int64_t>(p.R, 1);
    int64_t slots = 0, items;
    if (weights) {
        const int64_t per = int64_t(d.mtiles) * d.ntiles;
        // parts of at least so many rows that storing a part costs a fraction of them
        const int64_t least = 8 * std::min<int64_t>(p.K, NT);
        int64_t chunk = d.chunk;
        if (segments * per * cg < 8 * p.sms) chunk = std::max(least, ceil_to(ceil_to(p.R * per * cg, 4 * p.sms), KB) * KB);
        if (p.out_type != PT_F32) chunk = std::min(chunk, LONGEST);
        if (chunk < p.R) {
            d.chunk = chunk;
            d.add_by_start = segments > 2 * (p.R / chunk + 1);
            d.add_blocks = static_cast<int32_t>(std::min((d.add_by_start ? p.R / chunk + 1 : segments) * per, int64_t(INT32_MAX)));      // (more: too_many below)
            slots = 2 * (p.R / chunk + 1) * per;
        }
        items = (segments + p.R / d.chunk) * per;
    } else {
        items = d.row_tiles * d.mtiles;
        // parts of a tile: a cluster of 4 CTAs at most (8: slower than none by
        // half, one token's adapters 14.7 us against 9.0 with 4), which fit 27
        // of 32 SMs.  float32 parts are short enough to need no flushing.
        int64_t parts = 1;
        while (parts < 4 && items * cg * parts * 2 <= p.sms * 27 / 32 && d.part_blocks / (parts * 2) >= 4) parts *= 2;
        if (parts > 1 && ceil_to(d.part_blocks, parts) <= (p.type != PT_F32 ? LONGEST / KB : 16)) {
            d.part_blocks = static_cast<int32_t>(ceil_to(d.part_blocks, parts));
            d.parts = static_cast<int32_t>(parts);
            items *= parts;
        }
    }
    d.too_many = items > INT32_MAX;
    d.grid = static_cast<int32_t>(std::max<int64_t>(cg, std::min<int64_t>(items * cg, p.sms / cg * cg)));
    d.prefix_bytes = mode != PRODUCT_ADAPTERS && p.S > NEAR_SEGMENTS ? ceil_to((p.S + 1) * 8, 256) * 256 : 0;
    d.partial_bytes = ceil_to(slots * cg * NT * MT * 4, 256) * 256;
    d.staged = !d.empty && !weights && p.out_type != PT_F32 && d.parts == 1 && p.K > LONGEST;
    // gated: the accumulators hold the whole sum (see LONGEST, and KernelArgs::flush)
    d.fused = d.tensor && !d.staged && (p.type != PT_F32 || d.parts > 1 || d.part_blocks <= FLUSH_F32);
    if (d.staged) d.staged_bytes = ceil_to(p.R * p.N * 4, 256) * 256;
    if (d.pack_x) d.pack_x_bytes = ceil_to(packed_row(p.K, p.type) * p.R, 256) * 256;
    if (d.pack_w) {
        const MatShape m = w_shape(mode, p);
        d.pack_w_bytes = (halves_apart(mode, p) ? 2 * packed_row(m.cols / 2, p.type) : packed_row(m.cols, p.type)) * m.rows * m.mats;
    }
    return d;
}

// Requests of a row or two and of a low rank, or not many rows x ranks in all:
// every dot product is two warps' work and a search through the requests, while
// the tensor-core kernel has a tile per request, which costs the same for one
// row as for 16.  Whole calls, by rows / by tiles, us:
//   K = N = 4,096, rank 16: 96 requests x 1 row 22 / 38, 1,024 x 2 164 / 214,
//     4,096 x 2 671 / 722, 1,024 x 4 308 / 304, 4,096 x 4 1,314 / 1,055;
//   2,048, rank 64: 96 x 1 45 / 51, 96 x 2 67 / 64, 256 x 1 85 / 85, 256 x 2
//     106 / 85, 4,096 x 1 921 / 575, 4,096 x 4 3,519 / 1,565;
//   1,024, rank 8: 256 x 4 36 / 41, 1,024 x 4 97 / 92, 4,096 x 1 125 / 171,
//     4,096 x 2 229 / 211.
bool lora_by_rows(const ProductParams& p) {
    return p.S <= 4096 && p.R <= 4 * p.S && (p.R * p.N <= 16384 || (p.N <= 16 && p.R <= 2 * p.S));
}

namespace {

// halves 2: the two halves of each row of the matrices become rows of their own.
cudaError_t launch_pack(const void* src, int64_t ld, int64_t stride, const MatShape& m, int size, void* dst, int sms, cudaStream_t stream,
                        int halves = 1) {
    PackArgs a{};
    a.src = src;
    a.dst = static_cast<unsigned char*>(dst);
    a.ld = ld;
    a.stride = stride;
    a.rows = m.rows;
    a.cols = m.cols / halves;
    a.halves = halves;
    a.row_units = static_cast<int>(packed_row(a.cols, size == 4 ? PT_F32 : PT_F16) / 16);
    const int64_t rows = m.rows * m.mats * halves;
    a.units = rows * a.row_units;
    if (a.units == 0) return cudaSuccess;
    a.large = a.units > INT32_MAX;
    if (!a.large) {
        a.by_row = Divisor(static_cast<uint32_t>(a.row_units));
        a.by_mat = Divisor(static_cast<uint32_t>(m.rows * halves));
    }
    const int64_t blocks = std::min<int64_t>(ceil_to(a.units, 4 * 256), int64_t(sms) * 32);
    if (size == 4) pack_kernel<uint32_t><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    else pack_kernel<uint16_t><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lora_rows(const ProductParams& p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.R), static_cast<unsigned>(ceil_to(p.N, DOT_RANKS)));
    if (p.type == PT_F32) lora_rows_kernel<float><<<grid, DOT_RANKS * 64, 0, stream>>>(p);
    else if (p.type == PT_F16) lora_rows_kernel<__half><<<grid, DOT_RANKS * 64, 0, stream>>>(p);
    else lora_rows_kernel<__nv_bfloat16><<<grid, DOT_RANKS * 64, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_product(int mode, const ProductParams& given, const ProductPlan& plan, cudaStream_t stream) {
    ProductParams p = given;
    if (plan.empty) {
        // nothing to sum: zeros
        const size_t size = p.out_type == PT_F32 ? 4 : 2;
        if (mode == PRODUCT_WEIGHTS) return cudaMemsetAsync(p.out, 0, size * p.S * p.K * p.N, stream);
        if (mode == PRODUCT_GATED) {
            const size_t pre_size = p.pre_type == PT_F32 ? 4 : 2;
            const cudaError_t e = p.pre ? cudaMemset2DAsync(p.pre, pre_size * p.ldp, 0, pre_size * p.N, p.R, stream) : cudaSuccess;
            return e != cudaSuccess ? e : cudaMemset2DAsync(p.out, size * p.ldo, 0, size * (p.N / 2), p.R, stream);
        }
        return cudaMemset2DAsync(p.out, size * p.ldo, 0, size * p.N, p.R, stream);
    }
    unsigned char* packed = p.ws + plan.prefix_bytes + plan.partial_bytes + plan.staged_bytes;
    const int size = p.type == PT_F32 ? 4 : 2;
    float* const staged = reinterpret_cast<float*>(p.ws + plan.prefix_bytes + plan.partial_bytes);
    if (plan.staged) {
        p.out = staged;
        p.ldo = p.N;
        p.out_type = PT_F32;
    }
    if (plan.pack_x) {
        const cudaError_t e = launch_pack(p.x, p.ldx, 0, {1, p.R, p.K}, size, packed, p.sms, stream);
        if (e != cudaSuccess) return e;
        p.x = packed;
        p.ldx = packed_row(p.K, p.type) / size;
        packed += plan.pack_x_bytes;
    }
    int64_t half_w = p.trans ? p.N / 2 * p.ldw : p.N / 2;
    if (plan.pack_w) {
        const MatShape m = w_shape(mode, p);
        const int halves = halves_apart(mode, p) ? 2 : 1;
        const int64_t row = halves * packed_row(m.cols / halves, p.type);
        const cudaError_t e = launch_pack(p.w, p.ldw, p.stride_w, m, size, packed, p.sms, stream, halves);
        if (e != cudaSuccess) return e;
        half_w = p.trans ? p.N / 2 * (row / size) : row / 2 / size;
        p.w = packed;
        p.ldw = row / size;
        p.stride_w = m.rows * p.ldw;
    }
    KernelArgs a{};
    a.p = p;
    a.mtiles = plan.mtiles;
    a.ntiles = plan.ntiles;
    a.parts = plan.parts;
    a.part_blocks = plan.part_blocks;
    a.kblocks = static_cast<int32_t>(ceil_to(p.K, KB));
    const bool gated = mode == PRODUCT_GATED;
    a.box_rows = plan.narrow && p.R <= 32 * (mode == PRODUCT_FORWARD || gated ? p.S : 1) ? 16 : 64;
    a.a_rows = static_cast<int32_t>(gated ? std::min<int64_t>(MT / 2, ceil_to(p.N / 2, 16) * 16) : std::min<int64_t>(MT, ceil_to(p.N, 16) * 16));
    a.half_w = half_w;
    if (plan.parts > 1) a.flush = NEVER_FLUSH;                 // a part is short enough
    else if (p.type == PT_F32) a.flush = FLUSH_F32;
    else if (p.out_type != PT_F32) a.flush = NEVER_FLUSH;      // the sum is
    else a.flush = mode == PRODUCT_WEIGHTS ? 12 : LONGEST / KB;
    const int64_t out_step = mode == PRODUCT_WEIGHTS ? p.N : p.ldo;
    a.wide_rows = (gated ? p.N / 2 : p.N) % 8 == 0 && out_step % 8 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
    a.wide_pre = p.N / 2 % 8 == 0 && p.ldp % 8 == 0 && reinterpret_cast<uintptr_t>(p.pre) % 16 == 0;
    a.twin = p.type == PT_F32 && p.N <= MT / 2 && plan.parts == 1;
    a.chunk = plan.chunk;
    a.add_by_start = plan.add_by_start;
    a.row_tiles = plan.row_tiles;
    a.cols_m = gated ? p.N / 2 : p.N;
    a.cols_n = p.K;
    a.far = reinterpret_cast<int*>(p.ws);
    a.partials = reinterpret_cast<float*>(p.ws + plan.prefix_bytes);
    if (mode == PRODUCT_WEIGHTS) return launch_mode<PRODUCT_WEIGHTS>(a, plan, stream);
    if (gated) return plan.fused ? launch_mode<PRODUCT_GATED>(a, plan, stream) : cudaErrorInvalidConfiguration;
    const cudaError_t e = mode == PRODUCT_FORWARD ? launch_mode<PRODUCT_FORWARD>(a, plan, stream) : launch_mode<PRODUCT_ADAPTERS>(a, plan, stream);
    if (e != cudaSuccess || !plan.staged) return e;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(ceil_to(p.R * p.N, 1024), int64_t(p.sms) * 8));
    if (given.out_type == PT_F16) round_kernel<<<blocks, 256, 0, stream>>>(staged, static_cast<__half*>(given.out), p.R, p.N, given.ldo);
    else round_kernel<<<blocks, 256, 0, stream>>>(staged, static_cast<__nv_bfloat16*>(given.out), p.R, p.N, given.ldo);
    return cudaGetLastError();
}

}  // namespace segred

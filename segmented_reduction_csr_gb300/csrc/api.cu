// api.cu -- the C ABI of libsegreduce (declared in include/seg_reduce.h):
// argument checks, the host launch planner, the library-owned scratch cache
// and the kernel launch.  Nothing here reads device memory on the host.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "../../include/seg_reduce.h"
#include "seg_gated.cuh"
#include "seg_norm.cuh"
#include "seg_pick.cuh"
#include "seg_plan.cuh"
#include "seg_product.cuh"
#include "seg_rle.cuh"
#include "seg_scan.cuh"
#include "seg_scatter.cuh"
#include "seg_scratch.cuh"
#include "seg_seq.cuh"
#include "seg_sort.cuh"

using namespace segred;

namespace {

constexpr int32_t kVersion = 1 * 10000 + 0 * 100 + 0;
constexpr int kMaxDevices = 64;

// Self-test of the bounded waits: one thread waits, with the kernels' own
// wait_bounded_for, on an mbarrier phase that nothing completes; the wait
// runs out after limit_ns, ORs STATUS_CONSUMER_TIMEOUT into the status word
// and the kernel returns.  No copy is in flight and nothing else waits.
__global__ void selftest_wait_kernel(unsigned int* status, uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    mbar_init(&bar, 1);
    fence_mbarrier_init();
    (void)wait_bounded_for(&bar, 0, status, STATUS_CONSUMER_TIMEOUT, limit_ns);
}

// ---------------------------------------------------------------------------
// Per-device state: SM count, status word, kernels already configured.

struct DeviceState {
    bool init = false;
    int sm_count = 0;
    unsigned int* status = nullptr;
    std::map<const void*, bool> configured;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
std::map<std::pair<int, cudaStream_t>, Scratch> g_scratch;
// The deterministic scatter's sort buffers, offsets and gathered rows: a
// buffer of their own per (device, stream), so that the reduction it runs
// keeps its scratch (and its ticket words) to itself.
std::map<std::pair<int, cudaStream_t>, Scratch> g_sort_scratch;
// The products' scratch: a buffer of their own per (device, stream).
std::map<std::pair<int, cudaStream_t>, Scratch> g_product_scratch;

seg_status_t device_state(int dev, DeviceState** out) {
    if (dev < 0 || dev >= kMaxDevices) return SEG_ERR_CUDA;
    DeviceState& ds = g_dev[dev];
    if (!ds.init) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return SEG_ERR_CUDA;
        unsigned int* st = nullptr;
        if (cudaMalloc(&st, sizeof(unsigned int)) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_OUT_OF_MEMORY;
        }
        if (cudaMemset(st, 0, sizeof(unsigned int)) != cudaSuccess) return SEG_ERR_CUDA;
        ds.sm_count = sms;
        ds.status = st;
        ds.init = true;
    }
    *out = &ds;
    return SEG_OK;
}

// Scratch for (device, stream): grown on demand, zeroed when (re)allocated,
// stream-ordered so earlier work on the stream still sees the old buffer.
seg_status_t scratch_in(std::map<std::pair<int, cudaStream_t>, Scratch>& cache, int dev,
                        cudaStream_t stream, size_t bytes, Scratch** out) {
    Scratch& sc = cache[std::make_pair(dev, stream)];
    if (sc.bytes < bytes || sc.gen == UINT32_MAX) {
        size_t want = std::max<size_t>(bytes, size_t(1) << 20);
        want = std::max(want, sc.bytes);
        if (sc.ptr) cudaFreeAsync(sc.ptr, stream);
        sc.ptr = nullptr;
        sc.bytes = 0;
        if (cudaMallocAsync(&sc.ptr, want, stream) != cudaSuccess) {
            cudaGetLastError();
            sc.ptr = nullptr;
            return SEG_ERR_OUT_OF_MEMORY;
        }
        if (cudaMemsetAsync(sc.ptr, 0, want, stream) != cudaSuccess) return SEG_ERR_CUDA;
        sc.bytes = want;
        sc.gen = 0;
    }
    *out = &sc;
    return SEG_OK;
}

seg_status_t scratch_for(int dev, cudaStream_t stream, size_t bytes, Scratch** out) {
    return scratch_in(g_scratch, dev, stream, bytes, out);
}

// ---------------------------------------------------------------------------
// Scratch of products that are captured into a graph.  The graph keeps its
// address and may be replayed on any stream, beside other graphs that were
// captured from the same one, so every capture has buffers of its own: one
// per stream of the capture (whose calls follow one another in the graph too).
// They are ordinary device memory, and go back to a list of free ones when
// the graph and what was instantiated from it are gone.

struct GraphBuffer {
    int dev;
    size_t bytes;
    void* ptr;
    GraphBuffer* next;      // in the list of free ones
};
std::mutex g_free_mu;       // of the list alone: a graph may give a buffer back during any call of the runtime
GraphBuffer* g_free_buffers = nullptr;

void CUDART_CB give_back(void* buffer) {
    GraphBuffer* b = static_cast<GraphBuffer*>(buffer);
    std::lock_guard<std::mutex> lock(g_free_mu);
    b->next = g_free_buffers;
    g_free_buffers = b;
}

// The smallest free buffer of at least `bytes`, and at most four times as many; NULL: none.
GraphBuffer* take_free(int dev, size_t bytes) {
    std::lock_guard<std::mutex> lock(g_free_mu);
    GraphBuffer** best = nullptr;
    for (GraphBuffer** b = &g_free_buffers; *b; b = &(*b)->next)
        if ((*b)->dev == dev && (*b)->bytes >= bytes && (*b)->bytes / 4 <= bytes && (!best || (*b)->bytes < (*best)->bytes)) best = b;
    if (!best) return nullptr;
    GraphBuffer* b = *best;
    *best = b->next;
    return b;
}

struct CaptureScratch {
    unsigned long long id = 0;      // of the capture
    Scratch sc;
};
std::map<std::pair<int, cudaStream_t>, CaptureScratch> g_capture_scratch;

seg_status_t capture_scratch(int dev, cudaStream_t stream, unsigned long long id, cudaGraph_t graph, size_t bytes, Scratch** out) {
    CaptureScratch& cs = g_capture_scratch[std::make_pair(dev, stream)];
    if (cs.id != id) {
        cs.sc = Scratch();
        cs.id = id;
    }
    if (cs.sc.bytes < bytes) {      // (a smaller one stays with the calls before)
        const size_t want = std::max<size_t>(bytes, size_t(1) << 20);
        GraphBuffer* b = take_free(dev, want);
        if (!b) {
            b = new GraphBuffer{dev, want, nullptr, nullptr};
            // outside of the capture: what a capture allocates comes and goes with each replay
            cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
            cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
            if (e == cudaSuccess) {
                e = cudaMalloc(&b->ptr, want);
                cudaThreadExchangeStreamCaptureMode(&mode);
            }
            if (e != cudaSuccess) {
                cudaGetLastError();
                delete b;
                return SEG_ERR_OUT_OF_MEMORY;
            }
        }
        cudaUserObject_t owner;
        cudaError_t e = cudaUserObjectCreate(&owner, b, give_back, 1, cudaUserObjectNoDestructorSync);
        if (e == cudaSuccess) {
            e = cudaGraphRetainUserObject(graph, owner, 1, cudaGraphUserObjectMove);
            if (e != cudaSuccess) cudaUserObjectRelease(owner, 1);      // gives it back
        } else {
            give_back(b);
        }
        if (e != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        cs.sc.ptr = b->ptr;
        cs.sc.bytes = b->bytes;
    }
    *out = &cs.sc;
    return SEG_OK;
}

// Scratch of the products on `stream`, for what is enqueued or captured next.
seg_status_t product_scratch(int dev, cudaStream_t stream, size_t bytes, Scratch** out) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    cudaGraph_t graph = nullptr;
    if (cudaStreamGetCaptureInfo(stream, &status, &id, &graph, nullptr, nullptr, nullptr) != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    if (status != cudaStreamCaptureStatusNone) {
        if (status != cudaStreamCaptureStatusActive) return SEG_ERR_CUDA;      // a capture that has become invalid
        return capture_scratch(dev, stream, id, graph, bytes, out);
    }
    Scratch& sc = g_product_scratch[std::make_pair(dev, stream)];
    const bool there = grow_scratch(
        sc, bytes,
        [stream](void** ptr, size_t want) {
            if (cudaMallocAsync(ptr, want, stream) == cudaSuccess) return true;
            cudaGetLastError();
            return false;
        },
        [stream](void* ptr) { cudaFreeAsync(ptr, stream); });
    *out = &sc;
    return there ? SEG_OK : SEG_ERR_OUT_OF_MEMORY;
}

// ---------------------------------------------------------------------------
// Fixed scratch for seg_reduce_noalloc: static device memory, one array per
// device (a __device__ variable exists once in every context), so that call
// never allocates.  Its ticket words must read zero before the first launch;
// set-up clears them once per device.

static __device__ __align__(256) unsigned char g_fixed_scratch[SEG_NOALLOC_SCRATCH_BYTES];
static __device__ unsigned int g_fixed_status;   // device errors when the caller passes no word

constexpr int kMaxKernels = 128;   // compiled kernels: 3 dtypes x 3 ops x 2 offset types x 7 shapes

struct FixedState {
    bool init = false;
    int sm_count = 0;
    unsigned char* scratch = nullptr;
    unsigned int* status = nullptr;
    uint32_t gen = 0;
    const void* configured[kMaxKernels] = {};
    int n_configured = 0;
};

std::mutex g_fixed_mu;
FixedState g_fixed[kMaxDevices];

// First call on a device: SM count, the arrays' addresses, zeroed ticket
// words (waited for, so that every later launch on any stream sees zeros).
seg_status_t fixed_state(int dev, cudaStream_t stream, FixedState** out) {
    if (dev < 0 || dev >= kMaxDevices) return SEG_ERR_CUDA;
    FixedState& fs = g_fixed[dev];
    if (!fs.init) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return SEG_ERR_CUDA;
        void* scratch = nullptr;
        void* status = nullptr;
        if (cudaGetSymbolAddress(&scratch, g_fixed_scratch) != cudaSuccess ||
            cudaGetSymbolAddress(&status, g_fixed_status) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        const int64_t tickets = ticket_region_bytes(sms);
        if (tickets > int64_t(SEG_NOALLOC_SCRATCH_BYTES)) return SEG_ERR_SCRATCH_LIMIT;
        if (cudaMemsetAsync(scratch, 0, static_cast<size_t>(tickets), stream) != cudaSuccess ||
            cudaMemsetAsync(status, 0, sizeof(unsigned int), stream) != cudaSuccess ||
            cudaStreamSynchronize(stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        fs.sm_count = sms;
        fs.scratch = static_cast<unsigned char*>(scratch);
        fs.status = static_cast<unsigned int*>(status);
        fs.init = true;
    }
    *out = &fs;
    return SEG_OK;
}

// The offsets producers (run-length encoding, flags to offsets): the CTA
// count, scratch from the (device, stream) buffer past the ticket words
// (which these launches never touch), then the two launches.
seg_status_t run_producer(RleParams& p, int64_t n, int64_t* count, cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* ds = nullptr;
    seg_status_t st = device_state(dev, &ds);
    if (st != SEG_OK) return st;
    p.n = n;
    p.count = count;
    p.tiles = ceil_div(n, RLE_TILE);
    if (p.tiles > int64_t(INT32_MAX)) return SEG_ERR_UNSUPPORTED;   // tile indices stay 32-bit
    p.ctas = static_cast<int32_t>(std::min<int64_t>(
        p.tiles, std::min<int64_t>(int64_t(ds->sm_count) * RLE_CTAS_PER_SM, RLE_MAX_CTAS)));
    // scratch past the reduction's ticket words (which these launches never
    // touch): the per-CTA arrays, then the bitmap
    const int64_t ticket_bytes = ticket_region_bytes(ds->sm_count);
    Scratch* sc = nullptr;
    st = scratch_for(dev, stream,
                     static_cast<size_t>(ticket_bytes + RLE_CTA_SCRATCH + rle_tile_bytes(p.tiles)), &sc);
    if (st != SEG_OK) return st;
    int64_t* ws = reinterpret_cast<int64_t*>(static_cast<unsigned char*>(sc->ptr) + ticket_bytes);
    p.cta_count = ws;
    p.cta_first = ws + RLE_MAX_CTAS;
    p.tile_first = ws + 2 * RLE_MAX_CTAS;
    p.tile_count = reinterpret_cast<int32_t*>(p.tile_first + p.tiles);
    p.bitmap = reinterpret_cast<unsigned long long*>(
        reinterpret_cast<unsigned char*>(p.tile_first) + ((p.tiles * 12 + 255) / 256) * 256);
    static const char kProducerKey = 0;
    if (!ds->configured[&kProducerKey]) {
        if (configure_rle() != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        ds->configured[&kProducerKey] = true;
    }
    if (launch_rle(p, stream) != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

// Checks that the products share.  Nothing is launched when one fails.
int64_t product_size(seg_dtype_t dtype) { return dtype == SEG_F32 ? 4 : 2; }

bool bad_product_type(seg_dtype_t dtype) { return dtype != SEG_F32 && dtype != SEG_F16 && dtype != SEG_BF16; }

bool misaligned(const void* ptr, int64_t to) { return reinterpret_cast<uintptr_t>(ptr) % to != 0; }

seg_status_t check_product(seg_dtype_t dtype, int64_t num_rows, int64_t K, int64_t N, int64_t ldx,
                           const void* x, const void* offsets, seg_offset_dtype_t offsets_dtype, int64_t S) {
    if (bad_product_type(dtype)) return SEG_ERR_INVALID_ARGUMENT;
    if (offsets_dtype != SEG_OFF_U32 && offsets_dtype != SEG_OFF_I64) return SEG_ERR_INVALID_ARGUMENT;
    if (num_rows < 0 || K < 0 || N < 0 || S < 0 || ldx < K) return SEG_ERR_INVALID_ARGUMENT;
    if (num_rows > INT32_MAX - 4095 || S > (int64_t(1) << 30) || K > SEG_MAX_PRODUCT_COLUMNS || N > SEG_MAX_PRODUCT_COLUMNS)
        return SEG_ERR_UNSUPPORTED;
    if (num_rows > 0 && K > 0 && !x) return SEG_ERR_INVALID_ARGUMENT;
    if (S > 0 && !offsets) return SEG_ERR_INVALID_ARGUMENT;
    if (misaligned(x, product_size(dtype)) || misaligned(offsets, offsets_dtype == SEG_OFF_U32 ? 4 : 8))
        return SEG_ERR_INVALID_ARGUMENT;
    return SEG_OK;
}

bool bad_activation(seg_activation_t a) {
    return a != SEG_SILU && a != SEG_GELU && a != SEG_GELU_TANH && a != SEG_RELU && a != SEG_SIGMOID;
}

// What both passes of a norm take; offsets NULL: one segment of all rows.
seg_status_t check_norm(NormParams& p, const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t F, int64_t ldx, const void* weight,
                        seg_dtype_t weight_dtype, const void* offsets, seg_offset_dtype_t offsets_dtype, int64_t S) {
    if (!offsets && S != 1) return SEG_ERR_INVALID_ARGUMENT;
    const seg_status_t st = check_product(dtype, num_rows, F, 0, ldx, x, offsets ? offsets : x, offsets ? offsets_dtype : SEG_OFF_U32, offsets ? S : 0);
    if (st != SEG_OK) return st;
    if ((weight_dtype != dtype && weight_dtype != SEG_F32) || misaligned(weight, product_size(weight_dtype))) return SEG_ERR_INVALID_ARGUMENT;
    p.x = x;
    p.weight = weight;
    p.offsets = offsets;
    p.R = num_rows;
    p.F = F;
    p.S = S;
    p.ldx = ldx;
    p.type = dtype;
    p.weight_type = weight_dtype;
    p.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    return SEG_OK;
}

// No exception leaves a product's entry point (the containers allocate, the
// lock can fail).
template <class F>
seg_status_t guarded(F f) {
    try {
        return f();
    } catch (...) {
        return SEG_ERR_OUT_OF_MEMORY;
    }
}

// Enqueues one product on scratch that is large enough.
seg_status_t run_product(int mode, ProductParams p, cudaStream_t stream, Scratch* sc, DeviceState* ds) {
    p.sms = ds->sm_count;
    p.status = ds->status;
    p.ws = static_cast<unsigned char*>(sc->ptr);
    const ProductPlan plan = plan_product(mode, p);
    if (plan.too_many) return SEG_ERR_UNSUPPORTED;
    if (launch_product(mode, p, plan, stream) != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

seg_status_t run_product(int mode, ProductParams p, cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* ds = nullptr;
    seg_status_t st = device_state(dev, &ds);
    if (st != SEG_OK) return st;
    p.sms = ds->sm_count;
    Scratch* sc = nullptr;
    st = product_scratch(dev, stream, static_cast<size_t>(plan_product(mode, p).bytes()), &sc);
    return st != SEG_OK ? st : run_product(mode, p, stream, sc, ds);
}

}  // namespace

extern "C" {

seg_status_t seg_reduce_plan(seg_dtype_t dtype, int64_t F, int64_t num_values,
                             seg_offset_dtype_t offsets_dtype, int64_t num_segments, seg_op_t op,
                             uint64_t values_addr, int32_t sm_count, seg_plan_t* plan) {
    return plan_launch(dtype, F, num_values, offsets_dtype, num_segments, op, values_addr,
                       sm_count, plan);
}

seg_status_t seg_reduce(const void* values, seg_dtype_t dtype, int64_t F, int64_t num_values,
                        const void* offsets, seg_offset_dtype_t offsets_dtype,
                        int64_t num_segments, seg_op_t op, void* out, int64_t* out_arg,
                        seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int64_t S = num_segments;
    // Host-visible argument checks; nothing is launched when one fails.
    if (dtype != SEG_U32 && dtype != SEG_S32 && dtype != SEG_F32) return SEG_ERR_INVALID_ARGUMENT;
    if (offsets_dtype != SEG_OFF_U32 && offsets_dtype != SEG_OFF_I64) return SEG_ERR_INVALID_ARGUMENT;
    if (op != SEG_SUM && op != SEG_MIN && op != SEG_MAX && op != SEG_MEAN) return SEG_ERR_INVALID_ARGUMENT;
    if (F < 1 || num_values < 0 || S < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (op == SEG_MEAN && dtype != SEG_F32) return SEG_ERR_UNSUPPORTED;
    if (F > SEG_MAX_FEATURES) return SEG_ERR_UNSUPPORTED;
    if ((op == SEG_SUM || op == SEG_MEAN) && out_arg != nullptr) return SEG_ERR_INVALID_ARGUMENT;
    if (S == 0) return SEG_OK;
    if (!offsets || !out || (num_values > 0 && !values)) return SEG_ERR_INVALID_ARGUMENT;
    const size_t osz = offsets_dtype == SEG_OFF_U32 ? 4 : 8;
    if (reinterpret_cast<uintptr_t>(values) % 4 || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(offsets) % osz || reinterpret_cast<uintptr_t>(out_arg) % 8)
        return SEG_ERR_INVALID_ARGUMENT;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;

    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* ds = nullptr;
    seg_status_t st = device_state(dev, &ds);
    if (st != SEG_OK) return st;

    seg_plan_t pl;
    st = plan_launch(dtype, F, num_values, offsets_dtype, S, op,
                     reinterpret_cast<uint64_t>(values), ds->sm_count, &pl);
    if (st != SEG_OK) return st;

    const int kop = op == SEG_MIN ? OP_MIN : (op == SEG_MAX ? OP_MAX : OP_SUM);
    const int i64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    const void* fn = dtype == SEG_U32   ? pick_kernel_u32(kop, i64, pl.kernel_variant)
                     : dtype == SEG_S32 ? pick_kernel_s32(kop, i64, pl.kernel_variant)
                                        : pick_kernel_f32(kop, i64, pl.kernel_variant);
    if (!fn) return SEG_ERR_UNSUPPORTED;
    if (!ds->configured[fn]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(pl.smem_bytes)) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        ds->configured[fn] = true;
    }

    Scratch* sc = nullptr;
    st = scratch_for(dev, stream, static_cast<size_t>(pl.workspace_bytes), &sc);
    if (st != SEG_OK) return st;
    sc->gen += 1;

    Params prm;
    prm.values = values;
    prm.offsets = offsets;
    prm.out = out;
    prm.out_arg = (op == SEG_MIN || op == SEG_MAX) ? out_arg : nullptr;
    prm.N = num_values;
    prm.S = S;
    prm.F = static_cast<int32_t>(F);
    prm.G = F > 1 ? pl.vecs_per_thread : 1;   // rows kernel: column slices
    prm.K = pl.items_per_slot;
    prm.max_ends = pl.max_ends;
    prm.P = pl.grid;
    prm.mean = op == SEG_MEAN ? 1 : 0;
    const int64_t ticket_bytes = ticket_region_bytes(ds->sm_count);
    prm.ws_tickets = static_cast<unsigned long long*>(sc->ptr);
    prm.ws_parts = static_cast<unsigned char*>(sc->ptr) + ticket_bytes;
    prm.status = ds->status;
    prm.gen = sc->gen;

    void* args[] = {&prm};
    const cudaError_t e = cudaLaunchKernel(fn, dim3(pl.grid), dim3(pl.block), args,
                                           static_cast<size_t>(pl.smem_bytes), stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

const char* seg_reduce_strerror(seg_status_t status) {
    switch (status) {
        case SEG_OK: return "success";
        case SEG_ERR_INVALID_ARGUMENT: return "invalid argument";
        case SEG_ERR_UNSUPPORTED: return "unsupported combination of arguments";
        case SEG_ERR_OUT_OF_MEMORY: return "out of device memory for scratch";
        case SEG_ERR_CUDA: return "CUDA runtime error";
        case SEG_ERR_DEVICE_TIMEOUT: return "a bounded wait inside a kernel ran out";
        case SEG_ERR_SCRATCH_LIMIT: return "the call needs more scratch than the fixed no-allocation array holds";
        default: return "unknown status";
    }
}

seg_status_t seg_reduce_device_status(seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (cudaStreamSynchronize(stream) != cudaSuccess) return SEG_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    unsigned int* word = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        word = ds->status;
    }
    unsigned int h = 0;
    if (cudaMemcpy(&h, word, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return SEG_ERR_CUDA;
    if (h != 0 && cudaMemset(word, 0, sizeof(h)) != cudaSuccess) return SEG_ERR_CUDA;
    return h ? SEG_ERR_DEVICE_TIMEOUT : SEG_OK;
}

seg_status_t seg_reduce_noalloc(const void* values, seg_dtype_t dtype, int64_t F,
                                int64_t num_values, const void* offsets,
                                seg_offset_dtype_t offsets_dtype, int64_t num_segments, seg_op_t op,
                                void* out, int64_t* out_arg, unsigned int* status_word,
                                seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int64_t S = num_segments;
    // The same host-visible checks as seg_reduce; nothing is launched when one fails.
    if (dtype != SEG_U32 && dtype != SEG_S32 && dtype != SEG_F32) return SEG_ERR_INVALID_ARGUMENT;
    if (offsets_dtype != SEG_OFF_U32 && offsets_dtype != SEG_OFF_I64) return SEG_ERR_INVALID_ARGUMENT;
    if (op != SEG_SUM && op != SEG_MIN && op != SEG_MAX && op != SEG_MEAN) return SEG_ERR_INVALID_ARGUMENT;
    if (F < 1 || num_values < 0 || S < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (op == SEG_MEAN && dtype != SEG_F32) return SEG_ERR_UNSUPPORTED;
    if (F > SEG_MAX_FEATURES) return SEG_ERR_UNSUPPORTED;
    if ((op == SEG_SUM || op == SEG_MEAN) && out_arg != nullptr) return SEG_ERR_INVALID_ARGUMENT;
    if (S == 0) return SEG_OK;
    if (!offsets || !out || (num_values > 0 && !values)) return SEG_ERR_INVALID_ARGUMENT;
    const size_t osz = offsets_dtype == SEG_OFF_U32 ? 4 : 8;
    if (reinterpret_cast<uintptr_t>(values) % 4 || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(offsets) % osz || reinterpret_cast<uintptr_t>(out_arg) % 8 ||
        reinterpret_cast<uintptr_t>(status_word) % 4)
        return SEG_ERR_INVALID_ARGUMENT;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;

    std::lock_guard<std::mutex> lock(g_fixed_mu);
    FixedState* fs = nullptr;
    seg_status_t st = fixed_state(dev, stream, &fs);
    if (st != SEG_OK) return st;

    seg_plan_t pl;
    st = plan_launch(dtype, F, num_values, offsets_dtype, S, op,
                     reinterpret_cast<uint64_t>(values), fs->sm_count, &pl);
    if (st != SEG_OK) return st;
    if (pl.workspace_bytes > int64_t(SEG_NOALLOC_SCRATCH_BYTES)) return SEG_ERR_SCRATCH_LIMIT;

    const int kop = op == SEG_MIN ? OP_MIN : (op == SEG_MAX ? OP_MAX : OP_SUM);
    const int i64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    const void* fn = dtype == SEG_U32   ? pick_kernel_u32(kop, i64, pl.kernel_variant)
                     : dtype == SEG_S32 ? pick_kernel_s32(kop, i64, pl.kernel_variant)
                                        : pick_kernel_f32(kop, i64, pl.kernel_variant);
    if (!fn) return SEG_ERR_UNSUPPORTED;
    bool configured = false;
    for (int k = 0; k < fs->n_configured; ++k) configured = configured || fs->configured[k] == fn;
    if (!configured) {
        if (fs->n_configured >= kMaxKernels) return SEG_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(pl.smem_bytes)) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        fs->configured[fs->n_configured++] = fn;
    }
    // A new generation tag per call retires the previous call's ticket
    // counts; when the tag would wrap, the ticket words are cleared instead.
    if (fs->gen == UINT32_MAX) {
        if (cudaMemsetAsync(fs->scratch, 0, static_cast<size_t>(ticket_region_bytes(fs->sm_count)),
                            stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        fs->gen = 0;
    }
    fs->gen += 1;

    Params prm;
    prm.values = values;
    prm.offsets = offsets;
    prm.out = out;
    prm.out_arg = (op == SEG_MIN || op == SEG_MAX) ? out_arg : nullptr;
    prm.N = num_values;
    prm.S = S;
    prm.F = static_cast<int32_t>(F);
    prm.G = F > 1 ? pl.vecs_per_thread : 1;   // rows kernel: column slices
    prm.K = pl.items_per_slot;
    prm.max_ends = pl.max_ends;
    prm.P = pl.grid;
    prm.mean = op == SEG_MEAN ? 1 : 0;
    prm.ws_tickets = reinterpret_cast<unsigned long long*>(fs->scratch);
    prm.ws_parts = fs->scratch + ticket_region_bytes(fs->sm_count);
    prm.status = status_word != nullptr ? status_word : fs->status;
    prm.gen = fs->gen;

    void* args[] = {&prm};
    const cudaError_t e = cudaLaunchKernel(fn, dim3(pl.grid), dim3(pl.block), args,
                                           static_cast<size_t>(pl.smem_bytes), stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

seg_status_t seg_rle(const uint32_t* keys, int64_t n, uint32_t* values, uint32_t* lengths,
                     int64_t* offsets, int64_t* count, seg_stream_t stream) {
    if (n < 0 || n > int64_t(UINT32_MAX) || !count || (n > 0 && !keys)) return SEG_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(keys) % 4 || reinterpret_cast<uintptr_t>(values) % 4 ||
        reinterpret_cast<uintptr_t>(lengths) % 4 || reinterpret_cast<uintptr_t>(offsets) % 8 ||
        reinterpret_cast<uintptr_t>(count) % 8)
        return SEG_ERR_INVALID_ARGUMENT;
    RleParams p{};
    p.keys = keys;
    p.values = values;
    p.lengths = lengths;
    p.offsets = offsets;
    p.vec = reinterpret_cast<uintptr_t>(keys) % 16 == 0 ? 1 : 0;
    return run_producer(p, n, count, reinterpret_cast<cudaStream_t>(stream));
}

seg_status_t seg_flags_to_offsets(const uint8_t* flags, int64_t n, int64_t* offsets,
                                  int64_t* count, seg_stream_t stream) {
    if (n < 0 || !count || !offsets || (n > 0 && !flags)) return SEG_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(offsets) % 8 || reinterpret_cast<uintptr_t>(count) % 8)
        return SEG_ERR_INVALID_ARGUMENT;
    RleParams p{};
    p.flags = flags;
    p.flags_mode = 1;
    p.offsets = offsets;
    p.vec = reinterpret_cast<uintptr_t>(flags) % 16 == 0 ? 1 : 0;
    return run_producer(p, n, count, reinterpret_cast<cudaStream_t>(stream));
}

seg_status_t seg_reduce_sequential(const float* values, int64_t F, int64_t num_values,
                                   const void* offsets, seg_offset_dtype_t offsets_dtype,
                                   int64_t num_segments, seg_op_t op, float* out,
                                   seg_stream_t stream) {
    if (offsets_dtype != SEG_OFF_U32 && offsets_dtype != SEG_OFF_I64) return SEG_ERR_INVALID_ARGUMENT;
    if (op != SEG_SUM && op != SEG_MEAN) return SEG_ERR_INVALID_ARGUMENT;
    if (F < 1 || num_values < 0 || num_segments < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (F > SEG_MAX_FEATURES) return SEG_ERR_UNSUPPORTED;
    if (num_segments == 0) return SEG_OK;
    if (!offsets || !out || (num_values > 0 && !values)) return SEG_ERR_INVALID_ARGUMENT;
    const size_t osz = offsets_dtype == SEG_OFF_U32 ? 4 : 8;
    if (reinterpret_cast<uintptr_t>(values) % 4 || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(offsets) % osz)
        return SEG_ERR_INVALID_ARGUMENT;
    if (offsets_dtype == SEG_OFF_U32 && num_values > int64_t(UINT32_MAX)) return SEG_ERR_INVALID_ARGUMENT;
    if (ceil_div(num_segments * F, SEQ_NT) > int64_t(INT32_MAX)) return SEG_ERR_UNSUPPORTED;
    SeqParams p{};
    p.values = values;
    p.offsets = offsets;
    p.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    p.mean = op == SEG_MEAN ? 1 : 0;
    p.N = num_values;
    p.F = F;
    p.S = num_segments;
    p.out = out;
    if (launch_sequential(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

seg_status_t seg_scatter(const void* src, seg_dtype_t dtype, int64_t F, int64_t num_rows,
                         const int64_t* index, int64_t dim_size, seg_op_t op, void* out,
                         int64_t* out_arg, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype != SEG_U32 && dtype != SEG_S32 && dtype != SEG_F32) return SEG_ERR_INVALID_ARGUMENT;
    if (op != SEG_SUM && op != SEG_MIN && op != SEG_MAX && op != SEG_MEAN) return SEG_ERR_INVALID_ARGUMENT;
    if (F < 1 || num_rows < 0 || dim_size < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (op == SEG_MEAN && dtype != SEG_F32) return SEG_ERR_UNSUPPORTED;
    if (F > SEG_MAX_FEATURES) return SEG_ERR_UNSUPPORTED;
    if ((op == SEG_SUM || op == SEG_MEAN) && out_arg != nullptr) return SEG_ERR_INVALID_ARGUMENT;
    // rows are packed into 32 bits next to the value for max / min
    if (num_rows >= int64_t(UINT32_MAX)) return SEG_ERR_UNSUPPORTED;
    if (dim_size == 0) return SEG_OK;
    if (!out || (num_rows > 0 && (!src || !index))) return SEG_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(src) % 4 || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(index) % 8 || reinterpret_cast<uintptr_t>(out_arg) % 8)
        return SEG_ERR_INVALID_ARGUMENT;
    if (ceil_div(dim_size * F, 8) > int64_t(INT32_MAX)) return SEG_ERR_UNSUPPORTED;
    // one launch covers every element (no grid-stride loop): at most 2^30 CTAs
    if (ceil_div(num_rows * F, int64_t(SC_NT) * SC_ITEMS) > (int64_t(1) << 30)) return SEG_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* ds = nullptr;
    seg_status_t st = device_state(dev, &ds);
    if (st != SEG_OK) return st;
    ScatterParams p{};
    p.src = src;
    p.index = index;
    p.N = num_rows;
    p.F = F;
    p.D = dim_size;
    p.dtype = dtype == SEG_F32 ? 2 : (dtype == SEG_S32 ? 1 : 0);
    p.op = op == SEG_SUM ? 0 : (op == SEG_MIN ? 1 : (op == SEG_MAX ? 2 : 3));
    p.vec = (dtype == SEG_F32 && F % 4 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0 &&
             reinterpret_cast<uintptr_t>(out) % 16 == 0) ? 4 : 1;
    p.out = out;
    p.arg = (op == SEG_MIN || op == SEG_MAX) ? out_arg : nullptr;
    const int64_t need = (op == SEG_MIN || op == SEG_MAX) ? dim_size * F * 8 : (op == SEG_MEAN ? dim_size * 4 : 0);
    if (need > 0) {
        // scratch past the reduction's ticket words, which these launches never touch
        const int64_t ticket_bytes = ticket_region_bytes(ds->sm_count);
        Scratch* sc = nullptr;
        st = scratch_for(dev, stream, static_cast<size_t>(ticket_bytes + need), &sc);
        if (st != SEG_OK) return st;
        unsigned char* ws = static_cast<unsigned char*>(sc->ptr) + ticket_bytes;
        if (op == SEG_MEAN) p.count = reinterpret_cast<uint32_t*>(ws);
        else p.word = reinterpret_cast<unsigned long long*>(ws);
    }
    if (launch_scatter(p, stream) != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

seg_status_t seg_scatter_sorted(const void* src, seg_dtype_t dtype, int64_t F, int64_t num_rows,
                                const int64_t* index, int64_t dim_size, seg_op_t op, void* out,
                                int64_t* out_arg, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype != SEG_U32 && dtype != SEG_S32 && dtype != SEG_F32) return SEG_ERR_INVALID_ARGUMENT;
    if (op != SEG_SUM && op != SEG_MIN && op != SEG_MAX && op != SEG_MEAN) return SEG_ERR_INVALID_ARGUMENT;
    if (F < 1 || num_rows < 0 || dim_size < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (op == SEG_MEAN && dtype != SEG_F32) return SEG_ERR_UNSUPPORTED;
    if (F > SEG_MAX_FEATURES) return SEG_ERR_UNSUPPORTED;
    if ((op == SEG_SUM || op == SEG_MEAN) && out_arg != nullptr) return SEG_ERR_INVALID_ARGUMENT;
    // row numbers and keys are 32-bit
    if (num_rows >= int64_t(UINT32_MAX) || dim_size >= int64_t(UINT32_MAX)) return SEG_ERR_UNSUPPORTED;
    if (dim_size == 0) return SEG_OK;
    if (!out || (num_rows > 0 && (!src || !index))) return SEG_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(src) % 4 || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(index) % 8 || reinterpret_cast<uintptr_t>(out_arg) % 8)
        return SEG_ERR_INVALID_ARGUMENT;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    SortParams sp{};
    int64_t* offsets = nullptr;
    void* rows = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        // sort buffers, then offsets, then the gathered rows
        const int64_t sort_bytes = ceil_div(sort_scratch_bytes(num_rows), 256) * 256;
        const int64_t off_bytes = ceil_div((dim_size + 1) * 8, 256) * 256;
        const int64_t row_bytes = num_rows * F * 4;
        Scratch* sc = nullptr;
        st = scratch_in(g_sort_scratch, dev, stream, static_cast<size_t>(sort_bytes + off_bytes + row_bytes), &sc);
        if (st != SEG_OK) return st;
        unsigned char* ws = static_cast<unsigned char*>(sc->ptr);
        sp.index = index;
        sp.N = num_rows;
        sp.D = dim_size;
        sp.tiles = ceil_div(num_rows, SORT_TILE);
        for (int b = 0; b < 2; ++b) {
            sp.keys[b] = reinterpret_cast<uint32_t*>(ws) + b * num_rows;
            sp.vals[b] = reinterpret_cast<uint32_t*>(ws) + (2 + b) * num_rows;
        }
        sp.hist = reinterpret_cast<uint32_t*>(ws) + 4 * num_rows;
        sp.total = sp.hist + int64_t(SORT_RADIX) * sp.tiles;
        int bits = 0;
        for (int64_t d = dim_size; d > 0; d >>= 1) ++bits;   // keys go up to dim_size
        sp.passes = (bits + 7) / 8;
        offsets = reinterpret_cast<int64_t*>(ws + sort_bytes);
        rows = ws + sort_bytes + off_bytes;
        const uint32_t* sorted = sp.keys[(sp.passes - 1) & 1];
        const uint32_t* perm = sp.vals[(sp.passes - 1) & 1];
        if (launch_sort(sp, stream) != cudaSuccess ||
            launch_bucket_offsets(sorted, num_rows, dim_size, offsets, stream) != cudaSuccess ||
            launch_gather_rows(src, perm, num_rows, F, rows, stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
    }
    // the groups are contiguous now: the deterministic segmented reduction
    const seg_status_t st = seg_reduce(num_rows > 0 ? rows : nullptr, dtype, F, num_rows, offsets, SEG_OFF_I64,
                                       dim_size, op, out, out_arg, stream_);
    if (st != SEG_OK) return st;
    if (out_arg != nullptr && (op == SEG_MIN || op == SEG_MAX) && num_rows > 0) {
        // args name rows of the sorted copy: map them back to src's rows
        if (launch_map_args(out_arg, sp.vals[(sp.passes - 1) & 1], dim_size * F, stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
    }
    return SEG_OK;
}

seg_status_t seg_scan(const void* values, seg_dtype_t dtype, int64_t num_values, const void* offsets,
                      seg_offset_dtype_t offsets_dtype, int64_t num_segments, seg_op_t op,
                      int32_t exclusive, void* out, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype != SEG_U32 && dtype != SEG_S32 && dtype != SEG_F32) return SEG_ERR_INVALID_ARGUMENT;
    if (offsets_dtype != SEG_OFF_U32 && offsets_dtype != SEG_OFF_I64) return SEG_ERR_INVALID_ARGUMENT;
    if (op != SEG_SUM && op != SEG_MIN && op != SEG_MAX) return SEG_ERR_INVALID_ARGUMENT;
    if (exclusive != 0 && exclusive != 1) return SEG_ERR_INVALID_ARGUMENT;
    if (exclusive && op != SEG_SUM) return SEG_ERR_UNSUPPORTED;
    if (num_values < 0 || num_segments < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (num_values == 0) return SEG_OK;
    if (!values || !offsets || !out) return SEG_ERR_INVALID_ARGUMENT;
    const size_t osz = offsets_dtype == SEG_OFF_U32 ? 4 : 8;
    if (reinterpret_cast<uintptr_t>(values) % 4 || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(offsets) % osz)
        return SEG_ERR_INVALID_ARGUMENT;
    if (offsets_dtype == SEG_OFF_U32 && num_values > int64_t(UINT32_MAX)) return SEG_ERR_INVALID_ARGUMENT;
    const int64_t tiles = ceil_div(num_values, RS_TILE);
    if (tiles > int64_t(INT32_MAX)) return SEG_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* ds = nullptr;
    seg_status_t st = device_state(dev, &ds);
    if (st != SEG_OK) return st;
    // scratch past the reduction's ticket words: per-CTA words, then the bitmap;
    // the ticket is slot 0 of the ticket words, tagged with a new generation
    const int64_t ticket_bytes = ticket_region_bytes(ds->sm_count);
    const int64_t cta_bytes = int64_t(RS_MAX_CTAS) * (8 + 8 + 8 + 4 + 4 + 4);
    const int64_t bitmap_bytes = rs_bitmap_words(num_values) * 8;
    Scratch* sc = nullptr;
    st = scratch_for(dev, stream, static_cast<size_t>(ticket_bytes + cta_bytes + bitmap_bytes), &sc);
    if (st != SEG_OK) return st;
    sc->gen += 1;
    unsigned char* ws = static_cast<unsigned char*>(sc->ptr) + ticket_bytes;
    ScanParams p{};
    p.values = values;
    p.offsets = offsets;
    p.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    p.dtype = dtype == SEG_F32 ? 2 : (dtype == SEG_S32 ? 1 : 0);
    p.op = op == SEG_SUM ? 0 : (op == SEG_MIN ? 1 : 2);
    p.exclusive = exclusive;
    p.vec = reinterpret_cast<uintptr_t>(values) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 ? 1 : 0;
    p.N = num_values;
    p.S = num_segments;
    p.out = out;
    p.tiles = tiles;
    p.sm_count = ds->sm_count;
    p.gen = sc->gen;
    p.ticket = static_cast<unsigned long long*>(sc->ptr);
    p.cta_aggf = reinterpret_cast<PartPair*>(ws);
    p.carryf = p.cta_aggf + RS_MAX_CTAS;
    p.cta_first = reinterpret_cast<int64_t*>(p.carryf + RS_MAX_CTAS);
    p.cta_aggi = reinterpret_cast<uint32_t*>(p.cta_first + RS_MAX_CTAS);
    p.carryi = p.cta_aggi + RS_MAX_CTAS;
    p.cta_flag = reinterpret_cast<int32_t*>(p.carryi + RS_MAX_CTAS);
    p.bitmap = reinterpret_cast<unsigned long long*>(ws + cta_bytes);
    if (launch_scan(p, stream) != cudaSuccess) {
        cudaGetLastError();
        return SEG_ERR_CUDA;
    }
    return SEG_OK;
}

seg_status_t seg_matmul(const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t K, int64_t ldx,
                        const void* w, int64_t N, int64_t ldw, int64_t stride_w, int32_t transpose_w,
                        const void* offsets, seg_offset_dtype_t offsets_dtype, int64_t num_segments,
                        void* out, int64_t ldo, seg_stream_t stream) {
    const seg_status_t st = check_product(dtype, num_rows, K, N, ldx, x, offsets, offsets_dtype, num_segments);
    if (st != SEG_OK) return st;
    const int64_t wrows = transpose_w ? N : K, wcols = transpose_w ? K : N;
    if ((transpose_w != 0 && transpose_w != 1) || ldo < N || ldw < wcols || stride_w < 0) return SEG_ERR_INVALID_ARGUMENT;
    if (num_segments > 1 && wrows > 0 && stride_w < (wrows - 1) * ldw + wcols) return SEG_ERR_INVALID_ARGUMENT;
    if (num_rows == 0 || N == 0) return SEG_OK;
    if (!out || (num_segments > 0 && K > 0 && !w)) return SEG_ERR_INVALID_ARGUMENT;
    if (misaligned(w, product_size(dtype)) || misaligned(out, product_size(dtype))) return SEG_ERR_INVALID_ARGUMENT;
    ProductParams p{};
    p.x = x;
    p.w = w;
    p.offsets = offsets;
    p.out = out;
    p.R = num_rows;
    p.K = K;
    p.N = N;
    p.S = num_segments;
    p.ldx = ldx;
    p.ldw = ldw;
    p.stride_w = stride_w;
    p.ldo = ldo;
    p.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    p.trans = transpose_w;
    p.type = p.out_type = dtype;
    return guarded([&] { return run_product(PRODUCT_FORWARD, p, reinterpret_cast<cudaStream_t>(stream)); });
}

seg_status_t seg_matmul_grad_w(const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t K, int64_t ldx,
                               const void* dy, int64_t N, int64_t ldy, const void* offsets,
                               seg_offset_dtype_t offsets_dtype, int64_t num_segments, void* out,
                               seg_dtype_t out_dtype, seg_stream_t stream) {
    const seg_status_t st = check_product(dtype, num_rows, K, N, ldx, x, offsets, offsets_dtype, num_segments);
    if (st != SEG_OK) return st;
    if ((out_dtype != dtype && out_dtype != SEG_F32) || ldy < N) return SEG_ERR_INVALID_ARGUMENT;
    if (num_segments == 0 || K == 0 || N == 0) return SEG_OK;
    if (!out || (num_rows > 0 && !dy)) return SEG_ERR_INVALID_ARGUMENT;
    if (misaligned(dy, product_size(dtype)) || misaligned(out, product_size(out_dtype))) return SEG_ERR_INVALID_ARGUMENT;
    ProductParams p{};
    p.x = x;
    p.w = dy;
    p.offsets = offsets;
    p.out = out;
    p.R = num_rows;
    p.K = K;
    p.N = N;
    p.S = num_segments;
    p.ldx = ldx;
    p.ldw = ldy;
    p.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    p.type = dtype;
    p.out_type = out_dtype;
    return guarded([&] { return run_product(PRODUCT_WEIGHTS, p, reinterpret_cast<cudaStream_t>(stream)); });
}

seg_status_t seg_lora(const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t K, int64_t ldx,
                      const void* w, int64_t N, int64_t ldw, const void* a, const void* b,
                      int64_t num_adapters, int64_t rank, const void* offsets,
                      seg_offset_dtype_t offsets_dtype, int64_t num_segments, const int32_t* adapter,
                      const float* scale, void* out, int64_t ldo, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    seg_status_t st = check_product(dtype, num_rows, K, N, ldx, x, offsets, offsets_dtype, num_segments);
    if (st != SEG_OK) return st;
    if (ldw < K || ldo < N || num_adapters < 0 || rank < 1) return SEG_ERR_INVALID_ARGUMENT;
    if (rank > SEG_MAX_RANK || num_adapters > INT32_MAX) return SEG_ERR_UNSUPPORTED;
    if (num_rows == 0 || N == 0) return SEG_OK;
    if (!out || (K > 0 && !w)) return SEG_ERR_INVALID_ARGUMENT;
    if (num_segments > 0 && !adapter) return SEG_ERR_INVALID_ARGUMENT;
    if (num_adapters > 0 && (!b || (K > 0 && !a))) return SEG_ERR_INVALID_ARGUMENT;
    const int64_t size = product_size(dtype);
    if (misaligned(w, size) || misaligned(a, size) || misaligned(b, size) || misaligned(out, size) ||
        misaligned(adapter, 4) || misaligned(scale, 4))
        return SEG_ERR_INVALID_ARGUMENT;
    return guarded([&]() -> seg_status_t {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        // the products with a, scaled, in float32: u = scale * x a^T
        ProductParams pa{};
        pa.x = x;
        pa.w = a;
        pa.offsets = offsets;
        pa.index = adapter;
        pa.scale = scale;
        pa.R = num_rows;
        pa.K = K;
        pa.N = rank;
        pa.S = num_segments;
        pa.ldx = ldx;
        pa.ldw = K;
        pa.stride_w = rank * K;
        pa.ldo = rank;
        pa.L = num_adapters;
        pa.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
        pa.trans = 1;
        pa.type = dtype;
        pa.out_type = SEG_F32;
        pa.sms = ds->sm_count;
        // the shared product, to which the low-rank part is added
        ProductParams p = pa;
        p.w = w;
        p.scale = nullptr;
        p.out = out;
        p.N = N;
        p.ldw = ldw;
        p.stride_w = 0;
        p.ldo = ldo;
        p.out_type = dtype;
        p.b = b;
        p.rank = rank;
        const bool low = num_segments > 0 && num_adapters > 0;
        const bool by_rows = lora_by_rows(pa);
        const int64_t own = std::max(low && !by_rows ? plan_product(PRODUCT_FORWARD, pa).bytes() : 0, plan_product(PRODUCT_ADAPTERS, p).bytes());
        Scratch* sc = nullptr;
        st = product_scratch(dev, stream, static_cast<size_t>(own + num_rows * rank * 4), &sc);
        if (st != SEG_OK) return st;
        float* u = reinterpret_cast<float*>(static_cast<unsigned char*>(sc->ptr) + own);
        if (low) {
            pa.out = u;
            if (by_rows) {
                if (launch_lora_rows(pa, stream) != cudaSuccess) {
                    cudaGetLastError();
                    return SEG_ERR_CUDA;
                }
            } else {
                st = run_product(PRODUCT_FORWARD, pa, stream, sc, ds);
                if (st != SEG_OK) return st;
            }
            p.u = u;
            // beside a kernel of short dot products; the tensor-core one needs the
            // memory to itself (prompts of 8,193 rows: 238 us together, 211 one after the other)
            p.overlap = by_rows ? 1 : 0;
        }
        return run_product(PRODUCT_ADAPTERS, p, stream, sc, ds);
    });
}

seg_status_t seg_gated(const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t K, int64_t ldx,
                       const void* w, int64_t N, int64_t ldw, int64_t stride_w, int32_t transpose_w,
                       const void* offsets, seg_offset_dtype_t offsets_dtype, int64_t num_segments,
                       seg_activation_t activation, void* out, int64_t ldo, void* pre, seg_dtype_t pre_dtype,
                       int64_t ldp, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const seg_status_t checked = check_product(dtype, num_rows, K, N, ldx, x, offsets, offsets_dtype, num_segments);
    if (checked != SEG_OK) return checked;
    if (bad_activation(activation) || (pre && pre_dtype != dtype && pre_dtype != SEG_F32)) return SEG_ERR_INVALID_ARGUMENT;
    const int64_t wrows = transpose_w ? 2 * N : K, wcols = transpose_w ? K : 2 * N;
    if ((transpose_w != 0 && transpose_w != 1) || ldo < N || ldw < wcols || stride_w < 0 || (pre && ldp < 2 * N)) return SEG_ERR_INVALID_ARGUMENT;
    if (num_segments > 1 && wrows > 0 && stride_w < (wrows - 1) * ldw + wcols) return SEG_ERR_INVALID_ARGUMENT;
    if (2 * N > SEG_MAX_PRODUCT_COLUMNS) return SEG_ERR_UNSUPPORTED;
    if (num_rows == 0 || N == 0) return SEG_OK;
    if (!out || (num_segments > 0 && K > 0 && !w)) return SEG_ERR_INVALID_ARGUMENT;
    const int64_t size = product_size(dtype);
    if (misaligned(w, size) || misaligned(out, size) || (pre && misaligned(pre, product_size(pre_dtype)))) return SEG_ERR_INVALID_ARGUMENT;
    ProductParams p{};
    p.x = x;
    p.w = w;
    p.offsets = offsets;
    p.R = num_rows;
    p.K = K;
    p.N = 2 * N;
    p.S = num_segments;
    p.ldx = ldx;
    p.ldw = ldw;
    p.stride_w = stride_w;
    p.off64 = offsets_dtype == SEG_OFF_I64 ? 1 : 0;
    p.trans = transpose_w;
    p.type = dtype;
    return guarded([&]() -> seg_status_t {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        p.sms = ds->sm_count;
        p.out = out;
        p.ldo = ldo;
        p.out_type = dtype;
        p.pre = pre;
        p.ldp = ldp;
        p.pre_type = pre_dtype;
        p.activation = activation;
        const ProductPlan plan = plan_product(PRODUCT_GATED, p);
        Scratch* sc = nullptr;
        if (plan.fused || plan.empty) {
            st = product_scratch(dev, stream, static_cast<size_t>(plan.bytes()), &sc);
            return st != SEG_OK ? st : run_product(PRODUCT_GATED, p, stream, sc, ds);
        }
        // the products in float32 (where those are asked for: in their place), then the activation
        const bool in_place = pre && pre_dtype == SEG_F32;
        p.out_type = SEG_F32;
        p.ldo = in_place ? ldp : 2 * N;
        p.out = in_place ? pre : nullptr;
        const int64_t own = plan_product(PRODUCT_FORWARD, p).bytes();
        st = product_scratch(dev, stream, static_cast<size_t>(own + (in_place ? 0 : num_rows * 2 * N * 4)), &sc);
        if (st != SEG_OK) return st;
        if (!in_place) p.out = static_cast<unsigned char*>(sc->ptr) + own;
        st = run_product(PRODUCT_FORWARD, p, stream, sc, ds);
        if (st != SEG_OK) return st;
        GatedParams g{};
        g.pre = p.out;
        g.ldp = p.ldo;
        g.out = out;
        g.ldo = ldo;
        g.rounded = in_place ? nullptr : pre;
        g.ldr = ldp;
        g.R = num_rows;
        g.N = N;
        g.type = dtype;
        g.activation = activation;
        g.sms = ds->sm_count;
        if (launch_gated(g, stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        return SEG_OK;
    });
}

seg_status_t seg_gated_grad(const void* pre, seg_dtype_t pre_dtype, int64_t num_rows, int64_t N, int64_t ldp,
                            const void* dy, seg_dtype_t dtype, int64_t ldy, seg_activation_t activation, void* dpre, int64_t ldd,
                            seg_stream_t stream) {
    if (bad_product_type(dtype) || bad_activation(activation) || (pre_dtype != dtype && pre_dtype != SEG_F32)) return SEG_ERR_INVALID_ARGUMENT;
    if (num_rows < 0 || N < 0 || ldp < 2 * N || ldy < N || ldd < 2 * N) return SEG_ERR_INVALID_ARGUMENT;
    if (num_rows > INT32_MAX - 4095 || 2 * N > SEG_MAX_PRODUCT_COLUMNS) return SEG_ERR_UNSUPPORTED;
    if (num_rows == 0 || N == 0) return SEG_OK;
    const int64_t size = product_size(dtype);
    if (!pre || !dy || !dpre || misaligned(pre, product_size(pre_dtype)) || misaligned(dy, size) || misaligned(dpre, size)) return SEG_ERR_INVALID_ARGUMENT;
    GatedParams g{};
    g.pre = pre;
    g.ldp = ldp;
    g.dy = dy;
    g.ldy = ldy;
    g.out = dpre;
    g.ldo = ldd;
    g.R = num_rows;
    g.N = N;
    g.type = dtype;
    g.pre_type = pre_dtype;
    g.activation = activation;
    return guarded([&]() -> seg_status_t {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        const seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        g.sms = ds->sm_count;
        if (launch_gated_grad(g, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        return SEG_OK;
    });
}

seg_status_t seg_layer_norm(const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t F, int64_t ldx,
                            const void* weight, const void* bias, seg_dtype_t weight_dtype, const void* offsets,
                            seg_offset_dtype_t offsets_dtype, int64_t num_segments, float eps, void* out,
                            int64_t ldo, float* mean, float* rstd, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    NormParams p{};
    const seg_status_t checked = check_norm(p, x, dtype, num_rows, F, ldx, weight, weight_dtype, offsets, offsets_dtype, num_segments);
    if (checked != SEG_OK) return checked;
    if (ldo < F || !(eps >= 0.0f) || !(eps < INFINITY)) return SEG_ERR_INVALID_ARGUMENT;
    if (num_rows == 0 || F == 0) return SEG_OK;
    if (!out || misaligned(out, product_size(dtype)) || misaligned(bias, product_size(weight_dtype)) || misaligned(mean, 4) || misaligned(rstd, 4))
        return SEG_ERR_INVALID_ARGUMENT;
    p.bias = bias;
    p.out = out;
    p.ldo = ldo;
    p.mean = mean;
    p.rstd = rstd;
    p.eps = eps;
    return guarded([&]() -> seg_status_t {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        const seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        p.sms = ds->sm_count;
        if (launch_norm(p, plan_norm(false, p), stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        return SEG_OK;
    });
}

seg_status_t seg_layer_norm_grad(const void* x, seg_dtype_t dtype, int64_t num_rows, int64_t F, int64_t ldx,
                                 const void* dy, int64_t ldy, const float* mean, const float* rstd,
                                 const void* weight, seg_dtype_t weight_dtype, const void* offsets,
                                 seg_offset_dtype_t offsets_dtype, int64_t num_segments, void* dx, int64_t lddx,
                                 void* dweight, void* dbias, seg_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    NormParams p{};
    const seg_status_t checked = check_norm(p, x, dtype, num_rows, F, ldx, weight, weight_dtype, offsets, offsets_dtype, num_segments);
    if (checked != SEG_OK) return checked;
    if (ldy < F || (dx && lddx < F)) return SEG_ERR_INVALID_ARGUMENT;
    const int64_t size = product_size(dtype), wsize = product_size(weight_dtype);
    if (misaligned(dy, size) || misaligned(dx, size) || misaligned(dweight, wsize) || misaligned(dbias, wsize) || misaligned(mean, 4) ||
        misaligned(rstd, 4))
        return SEG_ERR_INVALID_ARGUMENT;
    if (F == 0) return SEG_OK;
    if (num_rows > 0 && (!dy || !mean || !rstd)) return SEG_ERR_INVALID_ARGUMENT;
    if (p.S == 0) dweight = dbias = nullptr;
    if (num_rows == 0) {
        for (void* sums : {dweight, dbias})
            if (sums && cudaMemsetAsync(sums, 0, static_cast<size_t>(p.S * F * wsize), stream) != cudaSuccess) {
                cudaGetLastError();
                return SEG_ERR_CUDA;
            }
        return SEG_OK;
    }
    if (!dx && !dweight && !dbias) return SEG_OK;
    p.dy = dy;
    p.ldy = ldy;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.out = dx;
    p.ldo = dx ? lddx : F;
    p.dweight = dweight;
    p.dbias = dbias;
    return guarded([&]() -> seg_status_t {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        p.sms = ds->sm_count;
        const NormPlan plan = plan_norm(true, p);
        Scratch* sc = nullptr;
        st = product_scratch(dev, stream, static_cast<size_t>(plan.sums_for(p) + plan.parts_for(p)), &sc);
        if (st != SEG_OK) return st;
        p.ws = static_cast<unsigned char*>(sc->ptr);
        if (launch_norm_grad(p, plan, stream) != cudaSuccess) {
            cudaGetLastError();
            return SEG_ERR_CUDA;
        }
        return SEG_OK;
    });
}

seg_status_t seg_selftest_wait_timeout(uint32_t limit_ms, seg_stream_t stream_) {
    if (limit_ms < 1 || limit_ms > 10000) return SEG_ERR_INVALID_ARGUMENT;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SEG_ERR_CUDA;
    unsigned int* status = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceState* ds = nullptr;
        const seg_status_t st = device_state(dev, &ds);
        if (st != SEG_OK) return st;
        status = ds->status;
    }
    selftest_wait_kernel<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream_)>>>(
        status, static_cast<uint64_t>(limit_ms) * 1000000ull);
    if (cudaGetLastError() != cudaSuccess) return SEG_ERR_CUDA;
    return SEG_OK;
}

int32_t seg_reduce_version(void) { return kVersion; }

}  // extern "C"

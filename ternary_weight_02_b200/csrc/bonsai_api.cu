// bonsai_api.cu -- the extern "C" boundary of libbonsai (declared in include/bonsai.h).
//
// Every entry point validates its arguments on the host before touching the
// GPU, returns a bonsai_status code, and launches asynchronously on the
// caller's stream.  Per-device state (device properties, the workspace) is
// created on first use and kept until bonsai_shutdown().
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>
#include <vector>

#include "../../include/bonsai.h"
#include "common.cuh"
#include "internal.h"

namespace bonsai {
namespace {

constexpr int kMaxDevices = 64;
// Sizes are int64 in the interface; kernels index with int64 but grid and
// per-row arithmetic assumes a row of K activations and a plane of N rows fit
// comfortably below these bounds.
constexpr int64_t kMaxDim = int64_t(1) << 31;

struct DeviceState {
    bool probed = false;
    int status = BONSAI_OK;  // BONSAI_ERR_ARCH if the device cannot run sm_100a code
    DeviceInfo info;
    void *ws_base = nullptr;
    size_t ws_bytes = 0;  // total allocation (counters + data)
    void *zb_base = nullptr;
    size_t zb_bytes = 0;  // the zero-initialised region
    // buffers that larger ones took the place of: captured calls still use them
    std::vector<void *> old_ws, old_zb;
};

std::mutex g_mutex;
DeviceState g_dev[kMaxDevices];
bool g_force_wait_timeouts = false;  // test hook (bonsai_debug_force_timeouts)

int probe_current(int *dev_out, DeviceState **st_out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return BONSAI_ERR_CUDA;
    }
    DeviceState &st = g_dev[dev];
    if (!st.probed) {
        DeviceInfo info;
        if (cudaDeviceGetAttribute(&info.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&info.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&info.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&info.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&info.l2_bytes, cudaDevAttrL2CacheSize, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&info.smem_reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess) {
            cudaGetLastError();
            return BONSAI_ERR_CUDA;
        }
        st.info = info;
        // the library is built for sm_100a only
        st.status = (info.major == 10 && info.minor == 0) ? BONSAI_OK : BONSAI_ERR_ARCH;
        st.probed = true;
    }
    st.info.force_wait_timeouts = g_force_wait_timeouts;
    *dev_out = dev;
    *st_out = &st;
    return st.status;
}

// Puts a buffer of at least `need` bytes, at least half as large again as the one it replaces
// (so that all replaced ones together hold about twice its bytes at most), in the place of
// *base, its first `zeroed` bytes (0: all) zero.  The old buffer stays, in `old`: captured
// calls hold its address, and work in flight may use it.
int grow_buffer(void **base, size_t *bytes, std::vector<void *> *old, size_t need, size_t zeroed) {
    try {
        old->reserve(old->size() + 1);
    } catch (...) {  // no exception leaves a C entry point
        return BONSAI_ERR_NOMEM;
    }
    size_t size = *bytes + *bytes / 2 > need ? *bytes + *bytes / 2 : need;
    void *p = nullptr;
    cudaError_t e = cudaMalloc(&p, size);
    if (e != cudaSuccess && size > need) {
        cudaGetLastError();
        size = need;
        e = cudaMalloc(&p, size);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return BONSAI_ERR_NOMEM;
    }
    if (cudaMemset(p, 0, zeroed == 0 ? size : zeroed) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        cudaFree(p);
        return BONSAI_ERR_CUDA;
    }
    if (*base) old->push_back(*base);
    *base = p;
    *bytes = size;
    return BONSAI_OK;
}

// Makes sure the current device's workspace holds at least data_bytes after the
// counter block.
int ensure_workspace(DeviceState &st, size_t data_bytes, size_t zeroed_bytes, Workspace *ws) {
    const size_t need = kCounterBytes + ((data_bytes + 255) / 256) * 256;
    // the zeroed region always holds at least the control words (the device status word)
    if (zeroed_bytes < kCtlRegionBytes) zeroed_bytes = kCtlRegionBytes;
    if (st.ws_bytes < need) {  // at least 64 MiB
        // counters must start at zero; the kernels keep them at zero afterwards
        const int rc = grow_buffer(&st.ws_base, &st.ws_bytes, &st.old_ws, need < (size_t(64) << 20) ? (size_t(64) << 20) : need,
                                   kCounterBytes);
        if (rc != BONSAI_OK) return rc;
    }
    if (st.zb_bytes < zeroed_bytes) {
        const int rc = grow_buffer(&st.zb_base, &st.zb_bytes, &st.old_zb,
                                   zeroed_bytes < (size_t(16) << 20) ? (size_t(16) << 20) : zeroed_bytes, 0);
        if (rc != BONSAI_OK) return rc;
    }
    ws->zeroed = static_cast<uint8_t *>(st.zb_base);
    ws->zeroed_bytes = st.zb_bytes;
    ws->counters = static_cast<unsigned int *>(st.ws_base);
    ws->data = static_cast<uint8_t *>(st.ws_base) + kCounterBytes;
    ws->data_bytes = st.ws_bytes - kCounterBytes;
    return BONSAI_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned_to(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int64_t kMaxHeads = 1 << 16, kMaxRopeDim = 1024, kMaxSequences = 1 << 20;

// A row stride of a matrix of heads: rows of `width` elements, 16-byte aligned.
bool row_stride_ok(int64_t ld, int64_t width) {
    return ld >= width && ld % 8 == 0 && ld <= (int64_t(1) << 40);
}

// The shape of a paged cache and of the query heads that use it.
int check_cache(int64_t Hq, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int kv_type) {
    if (kv_type != BONSAI_KV_F16 && kv_type != BONSAI_KV_E4M3) return BONSAI_ERR_ARG;
    if (Hkv < 1 || Hkv > kMaxHeads || Hq < 0 || Hq > kMaxHeads || Hq % Hkv != 0) return BONSAI_ERR_SHAPE;
    if (D != 64 && D != 128 && D != 256) return BONSAI_ERR_SHAPE;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return BONSAI_ERR_SHAPE;
    if (pages < 1 || pages >= kMaxDim || pages * Hkv >= kMaxDim) return BONSAI_ERR_SHAPE;
    return BONSAI_OK;
}

int check_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K <= 0 || K % kGroup != 0) return BONSAI_ERR_SHAPE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return BONSAI_ERR_SHAPE;
    return BONSAI_OK;
}

int check_fmt(int fmt) {
    return (fmt == BONSAI_FMT_PTQ1_0 || fmt == BONSAI_FMT_PQ2_0 || fmt == BONSAI_FMT_Q1_0 ||
            fmt == BONSAI_FMT_PQ2_0_G64)
               ? BONSAI_OK
               : BONSAI_ERR_FMT;
}

int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return BONSAI_OK;
    cudaGetLastError();
    return BONSAI_ERR_CUDA;
}

// Picks the kernel for AUTO, or checks an explicit choice.  Without the device (argument
// checks before the device is probed) AUTO assumes the integer GEMV's grid fits; callers
// resolve AUTO again with the device once it is known.
int resolve_algo(int algo, int64_t M, int64_t N, int64_t K, int fmt, const DeviceInfo *dev = nullptr) {
    if (algo == BONSAI_ALGO_AUTO) {
        if (M <= 3 && gemv_imma_supported(M, N, K, fmt) && (dev == nullptr || gemv_imma_grid_fits(N, K, *dev)))
            return BONSAI_ALGO_IMMA;
        if (M == 1 && gemv_supported(M, N, K, fmt)) return BONSAI_ALGO_GEMV;
        if (M <= 16 && skinny_supported(M, N, K, fmt)) return BONSAI_ALGO_SKINNY;
        if (gemm_supported(M, N, K, fmt)) return BONSAI_ALGO_GEMM;
        return BONSAI_ALGO_SIMPLE;
    }
    switch (algo) {
        case BONSAI_ALGO_SIMPLE: return algo;
        case BONSAI_ALGO_GEMV: return gemv_supported(M, N, K, fmt) ? algo : BONSAI_ERR_ALGO;
        case BONSAI_ALGO_SKINNY: return skinny_supported(M, N, K, fmt) ? algo : BONSAI_ERR_ALGO;
        case BONSAI_ALGO_GEMM: return gemm_supported(M, N, K, fmt) ? algo : BONSAI_ERR_ALGO;
        case BONSAI_ALGO_IMMA: return gemv_imma_supported(M, N, K, fmt) ? algo : BONSAI_ERR_ALGO;
        default: return BONSAI_ERR_ALGO;
    }
}

// As resolve_algo, for a call with an epilogue: the skinny kernel also takes larger batches there,
// in groups of 16 tokens that re-read the weights (from the L2, mostly), and the automatic choice
// compares the two kernels' estimated times.  PQ2_0, us, skinny in groups against GEMM:
//   1001 x 1024:  M = 32 8.3 / 27, M = 1024 19 / 38;  5120 x 5120: M = 64 30 / 34, M = 128 44 / 34;
//   5120 x 17408: M = 32 39 / 50, M = 64 87 / 50;  and where the estimates choose the slower one:
//   1024 x 4096:  M = 512 29 / 34 (the GEMM; g64 32.5 / 34.4).
int resolve_epilogue_algo(int algo, int64_t M, int64_t N, int64_t K, int fmt, const DeviceInfo *dev = nullptr) {
    if (M > 16 && skinny_groups_supported(M, N, K, fmt)) {
        if (algo == BONSAI_ALGO_SKINNY) return algo;
        if (algo == BONSAI_ALGO_AUTO && dev && skinny_groups_us(M, N, K, fmt) < gemm_epilogue_us(M, N, K, fmt, *dev))
            return BONSAI_ALGO_SKINNY;
    }
    return resolve_algo(algo, M, N, K, fmt, dev);
}

// Launches the chosen kernel (argument checks and the workspace are the caller's).
cudaError_t run_linear(int chosen, const uint16_t *x, const uint8_t *packed, const uint16_t *scales, uint16_t *y,
                       int64_t M, int64_t N, int64_t K, int fmt, int split_k, const Workspace &ws, cudaStream_t s,
                       const DeviceInfo &info, const Epilogue *epi = nullptr) {
    switch (chosen) {
        case BONSAI_ALGO_GEMV: return launch_gemv(x, packed, scales, y, N, K, fmt, split_k, ws, s, info, epi);
        case BONSAI_ALGO_SKINNY: return launch_skinny(x, packed, scales, y, M, N, K, fmt, split_k, ws, s, info, epi);
        case BONSAI_ALGO_GEMM: return launch_gemm(x, packed, scales, y, M, N, K, fmt, split_k, ws, s, info, 0, epi);
        case BONSAI_ALGO_IMMA: return launch_gemv_imma(x, packed, scales, y, M, N, K, fmt, ws, s, info, 0, epi);
        default: return launch_linear_simple(x, packed, scales, y, M, N, K, fmt, ws, s, info, epi);
    }
}

size_t workspace_for(int algo, int64_t M, int64_t N, int64_t K, int fmt, int split_k,
                     const DeviceInfo &info) {
    switch (algo) {
        case BONSAI_ALGO_GEMV: return gemv_workspace_bytes(N, K, fmt, split_k, info);
        case BONSAI_ALGO_SKINNY: return skinny_workspace_bytes(M, N, K, fmt, split_k, info);
        case BONSAI_ALGO_GEMM: return gemm_workspace_bytes(M, N, K, fmt, info);
        case BONSAI_ALGO_IMMA: return 0;
        default: return simple_workspace_bytes(M, N, K);
    }
}

}  // namespace

int current_device_info(DeviceInfo *out) {
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    const int rc = probe_current(&dev, &st);
    if (rc == BONSAI_OK) *out = st->info;
    return rc;
}

}  // namespace bonsai

using namespace bonsai;

extern "C" {

int bonsai_version(void) { return (0 << 16) | (1 << 8) | 0; }

const char *bonsai_status_string(int status) {
    switch (status) {
        case BONSAI_OK: return "ok";
        case BONSAI_ERR_NULL: return "a required pointer is NULL";
        case BONSAI_ERR_SHAPE: return "bad shape (negative size, K not a positive multiple of 128, or too large)";
        case BONSAI_ERR_FMT: return "unknown packing format";
        case BONSAI_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case BONSAI_ERR_CUDA: return "CUDA runtime call or kernel launch failed";
        case BONSAI_ERR_ARCH: return "current device is not an sm_100 (B200-class) GPU";
        case BONSAI_ERR_NOMEM: return "could not allocate the device workspace";
        case BONSAI_ERR_ALGO: return "the requested kernel cannot run this shape";
        case BONSAI_ERR_TOO_LARGE: return "the problem needs more than the fixed device scratch of the no-allocation entry point";
        case BONSAI_ERR_ARG: return "unknown activation, layout, scaling or cache type, or a parameter outside its range";
        default: return "unknown status";
    }
}

int bonsai_check_device(void) {
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    return probe_current(&dev, &st);
}

int64_t bonsai_packed_bytes(int fmt, int64_t N, int64_t K) {
    if (check_fmt(fmt) != BONSAI_OK) return BONSAI_ERR_FMT;
    if (check_shape(0, N, K) != BONSAI_OK) return BONSAI_ERR_SHAPE;
    if (fmt == BONSAI_FMT_PTQ1_0) return N * (K / kGroup) * kPtq1GroupBytes;
    if (fmt == BONSAI_FMT_Q1_0) return N * (K / 8);
    return N * (K / 4);
}

static int pack_common(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream,
                       int fmt) {
    int rc = check_shape(0, N, K);
    if (rc != BONSAI_OK) return rc;
    if (N == 0) return BONSAI_OK;
    if (!trits || !packed) return BONSAI_ERR_NULL;
    if (!aligned16(trits) || !aligned16(packed)) return BONSAI_ERR_ALIGN;
    int dev;
    DeviceState *st;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        rc = probe_current(&dev, &st);
    }
    if (rc != BONSAI_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (fmt == BONSAI_FMT_PTQ1_0) return cuda_status(launch_pack_ptq1(trits, packed, N, K, s, st->info));
    if (fmt == BONSAI_FMT_Q1_0) return cuda_status(launch_pack_q1(trits, packed, N, K, s, st->info));
    return cuda_status(launch_pack_pq2(trits, packed, N, K, s, st->info));
}

int bonsai_pack_ptq1(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream) {
    return pack_common(trits, packed, N, K, stream, BONSAI_FMT_PTQ1_0);
}

int bonsai_pack_pq2(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream) {
    return pack_common(trits, packed, N, K, stream, BONSAI_FMT_PQ2_0);
}

int bonsai_pack_q1(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream) {
    return pack_common(trits, packed, N, K, stream, BONSAI_FMT_Q1_0);
}

int bonsai_unpack(int fmt, const uint8_t *packed, int8_t *trits, int64_t N, int64_t K, void *stream) {
    int rc = check_fmt(fmt);
    if (rc != BONSAI_OK) return rc;
    rc = check_shape(0, N, K);
    if (rc != BONSAI_OK) return rc;
    if (N == 0) return BONSAI_OK;
    if (!trits || !packed) return BONSAI_ERR_NULL;
    if (!aligned16(trits) || !aligned16(packed)) return BONSAI_ERR_ALIGN;
    int dev;
    DeviceState *st;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        rc = probe_current(&dev, &st);
    }
    if (rc != BONSAI_OK) return rc;
    return cuda_status(launch_unpack(fmt, packed, trits, N, K, static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_hadamard128(const uint16_t *x, uint16_t *x_out, int64_t M, int64_t K, void *stream) {
    int rc = check_shape(M, 0, K);
    if (rc != BONSAI_OK) return rc;
    if (M == 0) return BONSAI_OK;
    if (!x || !x_out) return BONSAI_ERR_NULL;
    if (!aligned16(x) || !aligned16(x_out)) return BONSAI_ERR_ALIGN;
    int dev;
    DeviceState *st;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        rc = probe_current(&dev, &st);
    }
    if (rc != BONSAI_OK) return rc;
    return cuda_status(launch_hadamard_f16(x, x_out, M, K, static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_ternary_linear_algo(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                               uint16_t *y, int64_t M, int64_t N, int64_t K, int fmt, int algo,
                               int split_k, void *stream) {
    int rc = check_fmt(fmt);
    if (rc != BONSAI_OK) return rc;
    rc = check_shape(M, N, K);
    if (rc != BONSAI_OK) return rc;
    if (split_k < 0) return BONSAI_ERR_SHAPE;
    if (M == 0 || N == 0) return BONSAI_OK;
    if (!x || !packed || !scales || !y) return BONSAI_ERR_NULL;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(scales) || !aligned16(y))
        return BONSAI_ERR_ALIGN;
    int chosen = resolve_algo(algo, M, N, K, fmt);
    if (chosen < 0) return chosen;

    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    if (algo == BONSAI_ALGO_AUTO) chosen = resolve_algo(algo, M, N, K, fmt, &st->info);
    // the integer GEMV's hand-over between CTAs needs its whole grid on the GPU at once
    if (chosen == BONSAI_ALGO_IMMA && !gemv_imma_grid_fits(N, K, st->info)) return BONSAI_ERR_ALGO;
    Workspace ws;
    rc = ensure_workspace(*st, workspace_for(chosen, M, N, K, fmt, split_k, st->info),
                          chosen == BONSAI_ALGO_IMMA ? gemv_imma_zeroed_bytes(M, N, K) : 0, &ws);
    if (rc != BONSAI_OK) return rc;
    return cuda_status(run_linear(chosen, x, packed, scales, y, M, N, K, fmt, split_k, ws,
                                  static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_ternary_linear(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                          uint16_t *y, int64_t M, int64_t N, int64_t K, int fmt, void *stream) {
    return bonsai_ternary_linear_algo(x, packed, scales, y, M, N, K, fmt, BONSAI_ALGO_AUTO, 0,
                                      stream);
}

int bonsai_swiglu(const uint16_t *y, uint16_t *h, int64_t M, int64_t F, void *stream) {
    if (M < 0 || F < 0 || M > kMaxDim || F > kMaxDim) return BONSAI_ERR_SHAPE;
    if (M == 0 || F == 0) return BONSAI_OK;
    if (!y || !h) return BONSAI_ERR_NULL;
    if (!aligned16(y) || !aligned16(h)) return BONSAI_ERR_ALIGN;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    const int rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    return cuda_status(launch_swiglu(y, h, M, F, static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_ternary_linear_swiglu(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                                 uint16_t *h, int64_t M, int64_t F, int64_t K, int fmt, void *stream) {
    int rc = check_fmt(fmt);
    if (rc != BONSAI_OK) return rc;
    if (F < 0 || F > kMaxDim / 2) return BONSAI_ERR_SHAPE;
    const int64_t N = 2 * F;
    rc = check_shape(M, N, K);
    if (rc != BONSAI_OK) return rc;
    if (M == 0 || F == 0) return BONSAI_OK;
    if (!x || !packed || !scales || !h) return BONSAI_ERR_NULL;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(scales) || !aligned16(h))
        return BONSAI_ERR_ALIGN;
    int chosen = resolve_algo(BONSAI_ALGO_AUTO, M, N, K, fmt);
    if (chosen < 0) return chosen;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    chosen = resolve_algo(BONSAI_ALGO_AUTO, M, N, K, fmt, &st->info);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Workspace ws;
    if (chosen == BONSAI_ALGO_IMMA) {  // fused into the GEMV's epilogue
        rc = ensure_workspace(*st, 0, gemv_imma_zeroed_bytes(M, N, K), &ws);
        if (rc != BONSAI_OK) return rc;
        return cuda_status(launch_gemv_imma(x, packed, scales, h, M, N, K, fmt, ws, s, st->info, F));
    }
    if (chosen == BONSAI_ALGO_GEMM) {  // fused into the GEMM's epilogue
        rc = ensure_workspace(*st, workspace_for(chosen, M, N, K, fmt, 0, st->info), 0, &ws);
        if (rc != BONSAI_OK) return rc;
        return cuda_status(launch_gemm(x, packed, scales, h, M, N, K, fmt, 0, ws, s, st->info, F));
    }
    // otherwise: the linear layer into the tail of the workspace, then the SwiGLU kernel
    const size_t need = (workspace_for(chosen, M, N, K, fmt, 0, st->info) + 255) / 256 * 256;
    rc = ensure_workspace(*st, need + (size_t)M * (size_t)N * 2,
                          chosen == BONSAI_ALGO_IMMA ? gemv_imma_zeroed_bytes(M, N, K) : 0, &ws);
    if (rc != BONSAI_OK) return rc;
    uint16_t *y = reinterpret_cast<uint16_t *>(ws.data + need);
    Workspace inner = ws;
    inner.data_bytes = need;
    cudaError_t e = run_linear(chosen, x, packed, scales, y, M, N, K, fmt, 0, inner, s, st->info);
    if (e == cudaSuccess) e = launch_swiglu(y, h, M, F, s, st->info);
    return cuda_status(e);
}

int bonsai_ternary_linear_epilogue(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                                   const uint16_t *bias, const uint16_t *residual, uint16_t *y, int64_t M,
                                   int64_t N, int64_t K, int fmt, int act, int algo, int split_k, void *stream) {
    int rc = check_fmt(fmt);
    if (rc != BONSAI_OK) return rc;
    if (act < BONSAI_ACT_NONE || act > BONSAI_ACT_GELU_TANH) return BONSAI_ERR_ARG;
    rc = check_shape(M, N, K);
    if (rc != BONSAI_OK) return rc;
    if (split_k < 0) return BONSAI_ERR_SHAPE;
    if (M == 0 || N == 0) return BONSAI_OK;
    if (!x || !packed || !scales || !y) return BONSAI_ERR_NULL;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(scales) || !aligned16(y) || !aligned16(bias) ||
        !aligned16(residual))
        return BONSAI_ERR_ALIGN;
    int chosen = resolve_epilogue_algo(algo, M, N, K, fmt);
    if (chosen < 0) return chosen;
    if (algo == BONSAI_ALGO_GEMM && split_k == 3) return BONSAI_ERR_ALGO;  // (also without a device)

    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    if (algo == BONSAI_ALGO_AUTO) chosen = resolve_epilogue_algo(algo, M, N, K, fmt, &st->info);
    if (chosen == BONSAI_ALGO_GEMM && split_k == 3) return BONSAI_ERR_ALGO;
    if (chosen == BONSAI_ALGO_IMMA && !gemv_imma_grid_fits(N, K, st->info)) return BONSAI_ERR_ALGO;
    Workspace ws;
    rc = ensure_workspace(*st, workspace_for(chosen, M, N, K, fmt, split_k, st->info),
                          chosen == BONSAI_ALGO_IMMA ? gemv_imma_zeroed_bytes(M, N, K) : 0, &ws);
    if (rc != BONSAI_OK) return rc;
    Epilogue epi;
    epi.bias = bias;
    epi.residual = residual;
    epi.act = act;
    // without any of the three the call is the plain product
    const bool groups = chosen == BONSAI_ALGO_SKINNY && M > 16;  // only the epilogue's instance takes them
    const Epilogue *e = bias || residual || act != BONSAI_ACT_NONE || groups ? &epi : nullptr;
    return cuda_status(run_linear(chosen, x, packed, scales, y, M, N, K, fmt, split_k, ws,
                                  static_cast<cudaStream_t>(stream), st->info, e));
}

int bonsai_rope_frequencies(double *freqs, double *magnitude, int64_t R, double base, int scaling, double factor,
                            double original, double low, double high) {
    if (R < 0 || R % 2 != 0 || R > kMaxRopeDim) return BONSAI_ERR_SHAPE;
    if (scaling < BONSAI_ROPE_PLAIN || scaling > BONSAI_ROPE_BANDS) return BONSAI_ERR_ARG;
    if (!(base > 1) || !std::isfinite(base)) return BONSAI_ERR_ARG;
    if (scaling != BONSAI_ROPE_PLAIN && (!(factor >= 1) || !std::isfinite(factor))) return BONSAI_ERR_ARG;
    const bool banded = scaling == BONSAI_ROPE_YARN || scaling == BONSAI_ROPE_BANDS;
    if (banded && (!(original > 0) || !std::isfinite(original) || !(low > 0) || !(high > low) || !std::isfinite(high)))
        return BONSAI_ERR_ARG;
    if (!magnitude || (R > 0 && !freqs)) return BONSAI_ERR_NULL;
    *magnitude = scaling == BONSAI_ROPE_YARN ? 1.0 + 0.1 * std::log(factor) : 1.0;
    const double two_pi = 6.283185307179586476925;
    // one pair alone has frequency 1 whatever the base
    if (scaling == BONSAI_ROPE_NTK && R > 2) base *= std::pow(factor, (double)R / (double)(R - 2));
    // YaRN: the pair indices that turn `high` and `low` times over `original` positions
    double first = 0, last = 0;
    if (scaling == BONSAI_ROPE_YARN) {
        auto index_of = [&](double turns) { return R * std::log(original / (turns * two_pi)) / (2 * std::log(base)); };
        first = std::floor(index_of(high));
        last = std::ceil(index_of(low));
        first = first < 0 ? 0 : first;
        last = last > R - 1 ? R - 1 : last;
    }
    for (int64_t i = 0; i < R / 2; i++) {
        const double f = std::pow(base, -2.0 * (double)i / (double)R);
        double v = f;
        if (scaling == BONSAI_ROPE_LINEAR) v = f / factor;
        if (scaling == BONSAI_ROPE_YARN) {
            const double width = last - first < 1e-3 ? 1e-3 : last - first;
            double ramp = ((double)i - first) / width;
            ramp = ramp < 0 ? 0 : ramp > 1 ? 1 : ramp;
            v = f / factor * ramp + f * (1 - ramp);
        }
        if (scaling == BONSAI_ROPE_BANDS) {
            double s = (original * f / two_pi - low) / (high - low);  // turns over `original` positions
            s = s < 0 ? 0 : s > 1 ? 1 : s;
            v = f / factor * (1 - s) + f * s;
        }
        freqs[i] = v;
    }
    return BONSAI_OK;
}

int bonsai_rope(const uint16_t *x, uint16_t *out, const double *freqs, const int32_t *positions, int64_t T, int64_t H,
                int64_t D, int64_t R, int64_t ld_x, int64_t ld_out, float magnitude, int layout, void *stream) {
    if (layout != BONSAI_ROPE_HALF && layout != BONSAI_ROPE_INTERLEAVED) return BONSAI_ERR_ARG;
    if (T < 0 || T > kMaxDim || H < 0 || H > kMaxHeads || D <= 0 || D % 8 != 0 || D > kMaxRopeDim || R < 0 ||
        R % 2 != 0 || R > D)
        return BONSAI_ERR_SHAPE;
    if (!row_stride_ok(ld_x, H * D) || !row_stride_ok(ld_out, H * D)) return BONSAI_ERR_SHAPE;
    if (T > 1 && x != nullptr && x == out && ld_x != ld_out) return BONSAI_ERR_SHAPE;  // in place: the same rows
    if (T == 0 || H == 0) return BONSAI_OK;
    if (!x || !out || !positions || (R > 0 && !freqs)) return BONSAI_ERR_NULL;
    if (!aligned16(x) || !aligned16(out) || !aligned_to(freqs, 8) || !aligned_to(positions, 4)) return BONSAI_ERR_ALIGN;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    const int rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    const RopeArgs r = {freqs, positions, magnitude, (int)R, layout};
    return cuda_status(launch_rope(x, out, r, T, H, D, ld_x, ld_out, static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_rope_append(const uint16_t *qkv, uint16_t *q_out, void *k_cache, void *v_cache, const float *k_scale,
                       const float *v_scale, const double *freqs, const int32_t *positions, const int64_t *slots,
                       int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t R, int64_t ld_qkv, int64_t ld_q,
                       int64_t pages, int64_t page_size, float magnitude, int layout, int kv_type, void *stream) {
    if (layout != BONSAI_ROPE_HALF && layout != BONSAI_ROPE_INTERLEAVED) return BONSAI_ERR_ARG;
    int rc = check_cache(Hq, Hkv, D, pages, page_size, kv_type);
    if (rc != BONSAI_OK) return rc;
    if (T < 0 || T > kMaxDim || R < 0 || R % 2 != 0 || R > D) return BONSAI_ERR_SHAPE;
    if (!row_stride_ok(ld_qkv, (Hq + 2 * Hkv) * D) || !row_stride_ok(ld_q, Hq * D)) return BONSAI_ERR_SHAPE;
    if (T > 1 && Hq > 0 && qkv != nullptr && qkv == q_out && ld_qkv != ld_q) return BONSAI_ERR_SHAPE;
    if (T == 0) return BONSAI_OK;
    if (!qkv || (Hq > 0 && !q_out) || !k_cache || !v_cache || !positions || !slots || (R > 0 && !freqs))
        return BONSAI_ERR_NULL;
    if (kv_type == BONSAI_KV_E4M3 && (!k_scale || !v_scale)) return BONSAI_ERR_NULL;
    if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned_to(freqs, 8) ||
        !aligned_to(positions, 4) || !aligned_to(slots, 8) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4))
        return BONSAI_ERR_ALIGN;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    Workspace ws;  // the status word
    rc = ensure_workspace(*st, 0, 0, &ws);
    if (rc != BONSAI_OK) return rc;
    const RopeArgs r = {freqs, positions, magnitude, (int)R, layout};
    const KvCache c = {k_cache, v_cache, k_scale, v_scale, pages, (int)page_size, (int)Hkv, (int)D, kv_type};
    return cuda_status(launch_rope_append(qkv, q_out, c, r, slots, T, Hq, ld_qkv, ld_q, ws,
                                          static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_paged_attention(const uint16_t *q, const void *k_cache, const void *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *page_table, const int32_t *lengths, uint16_t *out,
                           float *lse, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t ld_q, int64_t ld_out,
                           int64_t pages, int64_t page_size, int64_t max_pages, int64_t window, float scale,
                           int kv_type, void *stream) {
    int rc = check_cache(Hq, Hkv, D, pages, page_size, kv_type);
    if (rc != BONSAI_OK) return rc;
    if (B < 0 || B > kMaxSequences || Hq < 1 || max_pages < 1 || max_pages > kMaxDim || window < 0)
        return BONSAI_ERR_SHAPE;
    if (!row_stride_ok(ld_q, Hq * D) || !row_stride_ok(ld_out, Hq * D)) return BONSAI_ERR_SHAPE;
    if (B == 0) return BONSAI_OK;
    if (!q || !k_cache || !v_cache || !page_table || !lengths || !out) return BONSAI_ERR_NULL;
    if (kv_type == BONSAI_KV_E4M3 && (!k_scale || !v_scale)) return BONSAI_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned_to(page_table, 4) ||
        !aligned_to(lengths, 4) || !aligned_to(lse, 4) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4))
        return BONSAI_ERR_ALIGN;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    Workspace ws;
    rc = ensure_workspace(*st, attention_workspace_bytes(D, Hq / Hkv, st->info), 0, &ws);
    if (rc != BONSAI_OK) return rc;
    const KvCache c = {const_cast<void *>(k_cache), const_cast<void *>(v_cache), k_scale, v_scale, pages,
                       (int)page_size, (int)Hkv, (int)D, kv_type};
    return cuda_status(launch_paged_attention(q, c, page_table, lengths, out, lse, B, Hq, ld_q, ld_out, max_pages,
                                              window, scale, ws, static_cast<cudaStream_t>(stream), st->info));
}

int bonsai_launch_count(int64_t M, int64_t N, int64_t K, int fmt, int algo, int split_k) {
    int rc = check_fmt(fmt);
    if (rc != BONSAI_OK) return rc;
    rc = check_shape(M, N, K);
    if (rc != BONSAI_OK) return rc;
    if (M == 0 || N == 0) return 0;
    int chosen = resolve_algo(algo, M, N, K, fmt);
    if (chosen < 0) return chosen;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    if (algo == BONSAI_ALGO_AUTO) chosen = resolve_algo(algo, M, N, K, fmt, &st->info);
    if (chosen == BONSAI_ALGO_IMMA && !gemv_imma_grid_fits(N, K, st->info)) return BONSAI_ERR_ALGO;
    switch (chosen) {
        case BONSAI_ALGO_GEMV: return gemv_launches(N, K, fmt, split_k, st->info);
        case BONSAI_ALGO_IMMA: return 1;  // the rotation and quantisation of x are fused
        case BONSAI_ALGO_GEMM: return 1;  // the rotation is the kernel's first phase
        case BONSAI_ALGO_SKINNY: {  // fused when its grid is resident at once
            const int n = skinny_launches(M, N, K, fmt, split_k, st->info);
            return n < 0 ? BONSAI_ERR_CUDA : n;
        }
        default: return 2;  // the rotation pass, then the kernel
    }
}

int bonsai_reserve(int64_t M, int64_t N, int64_t K) {
    int rc = check_shape(M, N, K);
    if (rc != BONSAI_OK) return rc;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    size_t need = simple_workspace_bytes(M, N, K), zneed = 0;
    for (int fmt = BONSAI_FMT_PTQ1_0; fmt <= BONSAI_FMT_PQ2_0_G64; fmt++) {
        size_t v;
        if (M <= 1 && gemv_supported(1, N, K, fmt)) {
            v = gemv_workspace_bytes(N, K, fmt, 0, st->info);
            need = v > need ? v : need;
        }
        for (int64_t m = 1; m <= 3 && m <= (M > 1 ? M : 1); m++)
            if (gemv_imma_supported(m, N, K, fmt)) {
                v = gemv_imma_zeroed_bytes(m, N, K);
                zneed = v > zneed ? v : zneed;
            }
        if (skinny_supported(M < 16 ? M : 16, N, K, fmt)) {
            v = skinny_workspace_bytes(M < 16 ? M : 16, N, K, fmt, 0, st->info);
            need = v > need ? v : need;
        }
        if (M > 16 && skinny_groups_supported(M < kSkinnyMaxTokens ? M : kSkinnyMaxTokens, N, K, fmt)) {
            v = skinny_workspace_bytes(M < kSkinnyMaxTokens ? M : kSkinnyMaxTokens, N, K, fmt, 0, st->info);
            need = v > need ? v : need;
        }
        if (gemm_supported(M, N, K, fmt)) {
            v = gemm_workspace_bytes(M, N, K, fmt, st->info);
            need = v > need ? v : need;
        }
    }
    Workspace ws;
    // + the tail in which a non-fused bonsai_ternary_linear_swiglu keeps its M x N output
    need = (need + 255) / 256 * 256 + (size_t)M * (size_t)N * 2;
    return ensure_workspace(*st, need, zneed, &ws);
}

int bonsai_device_status(void *stream, uint32_t *bits, int clear) {
    if (!bits) return BONSAI_ERR_NULL;
    *bits = 0;
    std::lock_guard<std::mutex> lock(g_mutex);
    int dev;
    DeviceState *st;
    int rc = probe_current(&dev, &st);
    if (rc != BONSAI_OK) return rc;
    if (!st->zb_base) return BONSAI_OK;  // no call has run on this device: nothing to report
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the status word, and those of calls captured before the region grew
    for (size_t i = 0; i <= st->old_zb.size(); i++) {
        unsigned int *word = static_cast<unsigned int *>(i == 0 ? st->zb_base : st->old_zb[i - 1]) + kCtlStatus;
        unsigned int host = 0;
        if (cudaMemcpyAsync(&host, word, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            (clear && cudaMemsetAsync(word, 0, sizeof(unsigned int), s) != cudaSuccess) ||
            cudaStreamSynchronize(s) != cudaSuccess) {
            cudaGetLastError();
            return BONSAI_ERR_CUDA;
        }
        *bits |= host;
    }
    return BONSAI_OK;
}

int bonsai_debug_force_timeouts(int enable) {
    std::lock_guard<std::mutex> lock(g_mutex);
    g_force_wait_timeouts = enable != 0;
    return BONSAI_OK;
}

void bonsai_shutdown(void) {
    std::lock_guard<std::mutex> lock(g_mutex);
    int current = -1;
    cudaGetDevice(&current);
    for (int d = 0; d < kMaxDevices; d++) {
        DeviceState &st = g_dev[d];
        if (!st.ws_base && !st.zb_base) continue;
        cudaSetDevice(d);
        cudaDeviceSynchronize();
        for (void *p : st.old_ws) cudaFree(p);
        for (void *p : st.old_zb) cudaFree(p);
        cudaFree(st.ws_base);  // (of a null pointer: nothing)
        cudaFree(st.zb_base);
        st.old_ws.clear();
        st.old_zb.clear();
        st.ws_base = st.zb_base = nullptr;
        st.ws_bytes = st.zb_bytes = 0;
    }
    if (current >= 0) cudaSetDevice(current);
    cudaGetLastError();
}

}  // extern "C"

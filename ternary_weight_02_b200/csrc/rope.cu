// rope.cu -- rotary positions, alone and with the append of keys and values to a paged cache.
//
// A pair (a, b) of a head at position p turns by the angle p * f of its frequency f:
// (a, b) -> magnitude * (a cos - b sin, b cos + a sin).  The angle is a product of up to
// 10^6 positions and a frequency: in FP32 its absolute error would pass the FP16 rounding
// of the result from a few thousand positions on, so it is formed in FP64, counted in turns
// and reduced to [-1/2, 1/2] there; sine and cosine of the rest are FP32.
//
// HBM-bound: 2 bytes read and 2 (an E4M3 entry 1) written per element.  A CTA takes a few
// tokens; each (token, pair) sine and cosine is computed once into shared memory and serves
// every head, while the first values are already on their way.  A thread's task is 8 pairs of
// one head, two 16-byte loads and stores half the rotated part apart in both layouts
// (neighbouring threads then move neighbouring 16 bytes).  When 8 pairs do not divide the
// rotated part (R % 16 != 0, !kWhole) the last task has fewer, and in the half layout the
// partners start inside a 16-byte chunk and move in words or halfwords.  What is not rotated is
// moved as it is, bits untouched.  8191 tokens of 48 heads of 128, device time in a graph of such
// calls: interleaved 32.1 us, 6.3 TB/s (96% of the measured copy), half 34.3 us (90%); with
// R = 126 interleaved 34.8, half 95 us.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace bonsai {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kAhead = 2;  // tasks of a thread whose loads are in flight together
constexpr int kMaxTokens = 8;  // of a CTA

struct Job {
    const uint16_t *x;
    uint16_t *out;
    int64_t ld_x, ld_out, T;
    int H, D;           // heads rotated: all of x, or (append) query and key heads
    int tokens;         // per CTA
    int per_head, rot;  // tasks of a rotated head; the first `rot` of them rotate
    int gap, base;      // then `gap` (0 or 1) for elements [R, base), the rest from base on
    int head_shift;     // log2 of per_head, or -1
    int copy_heads, per_copy;  // append: value heads and their tasks
    RopeArgs r;
    // append
    KvCache c;
    const int64_t *slots;
    int Hq, page_shift;
    unsigned int *status;
};

__device__ __forceinline__ float2 sincos_at(int pos, double freq, float magnitude) {
    double turns = (double)pos * freq * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float sn, cs;
    sincospif(2.f * (float)turns, &sn, &cs);
    return make_float2(magnitude * cs, magnitude * sn);
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
// value / scale, nearest even, saturated
__device__ __forceinline__ uint2 e4m3_of8(const float (&v)[8], float scale) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        u[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] / scale, v[2 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
}

// Up to 8 elements from element `at` of a row (16-byte aligned): whole chunks in one access.
template <bool kWhole>
__device__ __forceinline__ uint4 load8(const uint16_t *row, int at, int n) {
    const uint16_t *p = row + at;
    if (kWhole || (n == 8 && (at & 7) == 0)) return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (n == 8 && (at & 1) == 0) {
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool kWhole>
__device__ __forceinline__ void store8(uint16_t *row, int at, int n, const uint4 &u) {
    uint16_t *p = row + at;
    if (kWhole || (n == 8 && (at & 7) == 0)) {
        *reinterpret_cast<uint4 *>(p) = u;
        return;
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if (n == 8 && (at & 1) == 0) {
#pragma unroll
        for (int i = 0; i < 4; i++) reinterpret_cast<uint32_t *>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}
template <bool kWhole>
__device__ __forceinline__ void store8_e4m3(uint8_t *row, int at, int n, const float (&v)[8], float scale) {
    uint8_t *p = row + at;
    const uint2 u = e4m3_of8(v, scale);
    if (kWhole || (n == 8 && (at & 7) == 0)) {
        *reinterpret_cast<uint2 *>(p) = u;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (i < n) p[i] = (uint8_t)((i < 4 ? u.x : u.y) >> (8 * (i & 3)));
}

// kMode: 0 rotation alone, 1 append to an FP16 cache, 2 to an E4M3 cache.
// kWhole: R % 16 == 0.
template <int kMode, int kLayout, bool kWhole>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(Job job) {
    // cosines and sines: [token of the CTA][8 rot], the eight pairs of rotating task k as four
    // float4s at k, rot + k, 2 rot + k, 3 rot + k (neighbouring threads read neighbouring words)
    extern __shared__ __align__(16) float2 turn[];
    pdl_launch_dependents();
    pdl_wait();  // everything read or written here may belong to the previous kernel
    const int half = job.r.R / 2, turn_stride = 8 * job.rot;
    const int chunks = (half + 3) >> 2;  // interleaved: 16-byte chunks with pairs
    const int64_t t0 = (int64_t)blockIdx.x * job.tokens;
    const int nt = (int)(job.T - t0 < job.tokens ? job.T - t0 : job.tokens);
    const int rot_tasks = job.H * job.per_head, per_token = rot_tasks + job.copy_heads * job.per_copy;
    const int total = nt * per_token;

    struct Task {
        int token, head;
        int at0, n0, at1, n1;  // first elements of the two chunks in the head, and their elements (0: none)
        int task;              // which of the head's rotating tasks, or -1: a copy
    };
    auto task_of = [&](int u) {
        Task k;
        k.token = 0;
        if (job.tokens > 1) {
            k.token = u / per_token;
            u -= k.token * per_token;
        }
        int i;
        bool value = false;
        if (kMode == 0 || u < rot_tasks) {
            k.head = job.head_shift >= 0 ? u >> job.head_shift : u / job.per_head;
            i = u - k.head * job.per_head;
        } else {
            u -= rot_tasks;
            k.head = u / job.per_copy;
            i = u - k.head * job.per_copy;
            k.head += job.H;
            value = true;
        }
        k.task = -1;
        k.n0 = k.n1 = 8;
        if (!value && i < job.rot) {
            k.task = i;
            // half: elements 8i .. and their partners; interleaved: 16-byte chunks i and rot + i
            k.at0 = 8 * i;
            k.at1 = kLayout == 0 ? 8 * i + half : 8 * (job.rot + i);
            if (!kWhole && kLayout == 0) k.n0 = k.n1 = half - 8 * i < 8 ? half - 8 * i : 8;
            if (!kWhole && kLayout == 1 && job.rot + i >= chunks) k.n1 = 0;
        } else if (!kWhole && !value && i < job.rot + job.gap) {
            k.at0 = k.at1 = job.r.R, k.n0 = job.base - job.r.R, k.n1 = 0;
        } else {
            k.at0 = value ? 16 * i : job.base + 16 * (i - job.rot - job.gap);
            k.at1 = k.at0 + 8;
            if (k.at1 >= job.D) k.n1 = 0;
        }
        return k;
    };
    auto row_of = [&](const Task &k) { return job.x + (t0 + k.token) * job.ld_x + (int64_t)k.head * job.D; };

    // key or value head of a task (append), past the query heads
    auto kv_head = [&](const Task &k) { return k.head < job.H ? k.head - job.Hq : k.head - job.H; };

    uint4 w0[kAhead], w1[kAhead];
    float sc[kAhead];
    auto load = [&](int base) {
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int u = base + j * (int)blockDim.x + (int)threadIdx.x;
            if (u >= total) continue;
            const Task k = task_of(u);
            const uint16_t *row = row_of(k);
            w0[j] = load8<kWhole>(row, k.at0, k.n0);
            if (k.n1 > 0) w1[j] = load8<kWhole>(row, k.at1, k.n1);
            sc[j] = 1.f;
            if (kMode == 2 && k.head >= job.Hq)
                sc[j] = __ldcg((k.head < job.H ? job.c.k_scale : job.c.v_scale) + kv_head(k));
        }
    };
    // the slots first, the barrier below waits for them (4096 tokens of 448 tasks: 23.9 us, 26.6
    // with the slots behind the turns; E4M3 25.8 and 28.7)
    int64_t slot = 0;
    if (kMode != 0 && (int)threadIdx.x < nt) slot = __ldcg(job.slots + t0 + threadIdx.x);
    load(0);
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int token = i / half;
        const int pair = i - token * half;
        int task, quarter;  // of the pair's float4
        if (kLayout == 0) {
            task = pair >> 3, quarter = (pair & 7) >> 1;
        } else {
            const int chunk = pair >> 2, second = chunk >= job.rot;
            task = second ? chunk - job.rot : chunk, quarter = 2 * second + ((pair & 3) >> 1);
        }
        turn[token * turn_stride + (quarter * job.rot + task) * 2 + (pair & 1)] =
            sincos_at(__ldcg(job.r.positions + t0 + token), __ldcg(job.r.freqs + pair), job.r.magnitude);
    }
    // row of the tokens' entries in the pools' first head (or -1), in rows of D elements
    __shared__ int64_t entry[kMaxTokens];
    if (kMode != 0 && (int)threadIdx.x < nt) {
        if (slot >= job.c.pages * job.c.page_size) atomicOr(job.status, kDevStatusCacheRange);
        const bool in = slot >= 0 && slot < job.c.pages * job.c.page_size;
        entry[threadIdx.x] = in ? (((slot >> job.page_shift) * job.c.kv_heads) << job.page_shift) + (slot & (job.c.page_size - 1)) : -1;
    }
    __syncthreads();
    auto finish = [&](const Task &k, const uint4 &c0, const uint4 &c1, float scale) {
        float a[8], b[8];
        unpack8(c0, a);
        unpack8(c1, b);
        uint4 u0 = c0, u1 = c1;  // what is not rotated keeps its bits, a NaN's too
        if (k.task >= 0) {
            const float4 *cs = reinterpret_cast<const float4 *>(turn + k.token * turn_stride) + k.task;
            float2 f[8];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float4 v = cs[i * job.rot];
                f[2 * i] = make_float2(v.x, v.y), f[2 * i + 1] = make_float2(v.z, v.w);
            }
            if constexpr (kLayout == 0) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float p = a[i], q = b[i];
                    a[i] = p * f[i].x - q * f[i].y;
                    b[i] = q * f[i].x + p * f[i].y;
                }
            } else {
                auto rotate = [&](float (&v)[8], const float2 *g, int first) {  // pairs first .. of a chunk
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (!kWhole && first + i >= half) continue;  // (elements that are not rotated, for an E4M3 entry)
                        const float p = v[2 * i], q = v[2 * i + 1];
                        v[2 * i] = p * g[i].x - q * g[i].y;
                        v[2 * i + 1] = q * g[i].x + p * g[i].y;
                    }
                };
                rotate(a, f, 4 * k.task);
                rotate(b, f + 4, 4 * (job.rot + k.task));
            }
            u0 = pack8(a), u1 = pack8(b);
            if (!kWhole && kLayout == 1) {
                auto rest = [&](uint4 &u, const uint4 &c, int first) {  // pairs of the chunk past the rotated ones
                    if (first + 0 >= half) u.x = c.x;
                    if (first + 1 >= half) u.y = c.y;
                    if (first + 2 >= half) u.z = c.z;
                    if (first + 3 >= half) u.w = c.w;
                };
                rest(u0, c0, 4 * k.task);
                rest(u1, c1, 4 * (job.rot + k.task));
            }
        }
        auto put16 = [&](uint16_t *row) {
            store8<kWhole>(row, k.at0, k.n0, u0);
            if (k.n1 > 0) store8<kWhole>(row, k.at1, k.n1, u1);
        };
        if (kMode == 0 || k.head < job.Hq) {
            put16(job.out + (t0 + k.token) * job.ld_out + (int64_t)k.head * job.D);
        } else {
            const int64_t first = entry[k.token], at = (first + ((int64_t)kv_head(k) << job.page_shift)) * job.D;
            if (first >= 0) {
                void *pool = k.head < job.H ? job.c.k : job.c.v;
                if constexpr (kMode == 1) {
                    put16(static_cast<uint16_t *>(pool) + at);
                } else {
                    uint8_t *row = static_cast<uint8_t *>(pool) + at;
                    store8_e4m3<kWhole>(row, k.at0, k.n0, a, scale);
                    if (k.n1 > 0) store8_e4m3<kWhole>(row, k.at1, k.n1, b, scale);
                }
            }
        }
    };
    for (int base = 0; base < total; base += kAhead * (int)blockDim.x) {
        if (base > 0) load(base);
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int u = base + j * (int)blockDim.x + (int)threadIdx.x;
            if (u < total) finish(task_of(u), w0[j], w1[j], sc[j]);
        }
    }
}

// Tasks, CTAs and shared memory of a job, and its launch.
template <int kMode>
cudaError_t launch(Job &job, cudaStream_t s, const DeviceInfo &dev) {
    const int R = job.r.R, D = job.D;
    const bool whole = R % 16 == 0, halves = job.r.layout == 0;
    const int chunks = (R / 2 + 3) / 4;
    job.rot = halves ? (R / 2 + 7) / 8 : (chunks + 1) / 2;
    job.base = halves ? (R + 7) / 8 * 8 : 8 * chunks;
    job.gap = halves && R % 8 != 0;
    // in place, what is not rotated already is where it belongs
    const bool in_place = kMode == 0 && job.x == job.out;
    job.per_head = job.rot + (in_place ? 0 : job.gap + (D - job.base + 15) / 16);
    if (in_place) job.gap = 0;
    job.per_copy = (D + 15) / 16;
    const int64_t per_token = (int64_t)job.H * job.per_head + (int64_t)job.copy_heads * job.per_copy;
    if (per_token == 0) return cudaSuccess;
    // several small tokens per CTA, as long as every SM still gets four CTAs
    int64_t tokens = 256 / per_token;
    const int64_t spread = job.T / (4 * (int64_t)dev.sm_count);
    tokens = tokens < spread ? tokens : spread;
    tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
    job.tokens = (int)tokens;
    // Few tokens: every task its own thread (32 tokens of 448 tasks: 2.9 us with 512 threads, 4.3
    // with 128).  Many: four tasks per thread keep more loads in flight per CTA and fewer warps at
    // its barrier (8191 tokens of 384 tasks: 34.3 us with 128 threads, 39.3 with 256).
    int64_t threads = job.T < 2 * (int64_t)dev.sm_count ? per_token * tokens : 128;
    threads = threads > kMaxThreads ? kMaxThreads : threads < 64 ? 64 : (threads + 31) / 32 * 32;
    job.head_shift = -1;
    for (int i = 0; i < 16; i++)
        if (job.per_head == 1 << i) job.head_shift = i;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((job.T + tokens - 1) / tokens));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)tokens * (size_t)(8 * job.rot) * sizeof(float2);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (whole)
        return cudaLaunchKernelEx(&cfg, halves ? rope_kernel<kMode, 0, true> : rope_kernel<kMode, 1, true>, job);
    return cudaLaunchKernelEx(&cfg, halves ? rope_kernel<kMode, 0, false> : rope_kernel<kMode, 1, false>, job);
}

}  // namespace

cudaError_t launch_rope(const uint16_t *x, uint16_t *out, const RopeArgs &r, int64_t T, int64_t H, int64_t D,
                        int64_t ld_x, int64_t ld_out, cudaStream_t s, const DeviceInfo &dev) {
    Job job = {};
    job.x = x, job.out = out, job.ld_x = ld_x, job.ld_out = ld_out, job.T = T;
    job.H = (int)H, job.D = (int)D, job.Hq = (int)H;
    job.r = r;
    return launch<0>(job, s, dev);
}

cudaError_t launch_rope_append(const uint16_t *qkv, uint16_t *q_out, const KvCache &c, const RopeArgs &r,
                               const int64_t *slots, int64_t T, int64_t Hq, int64_t ld_qkv, int64_t ld_q,
                               const Workspace &ws, cudaStream_t s, const DeviceInfo &dev) {
    Job job = {};
    job.x = qkv, job.out = q_out, job.ld_x = ld_qkv, job.ld_out = ld_q, job.T = T;
    job.H = (int)Hq + c.kv_heads, job.D = c.head_dim, job.Hq = (int)Hq, job.copy_heads = c.kv_heads;
    job.r = r;
    job.c = c;
    job.slots = slots;
    while ((1 << job.page_shift) < c.page_size) job.page_shift++;
    job.status = reinterpret_cast<unsigned int *>(ws.zeroed) + kCtlStatus;
    return c.type == 0 ? launch<1>(job, s, dev) : launch<2>(job, s, dev);
}

}  // namespace bonsai

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
// (neighbouring threads then move neighbouring 16 bytes); when 8 pairs do not divide the
// rotated part (R % 16 != 0) a task is one pair.  8191 tokens of 48 heads of 128: 34.8 us,
// 5.79 TB/s (89% of the measured copy); with one pair per task 100 us.
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
__device__ __forceinline__ uint8_t e4m3_of(float v, float scale) {
    return __nv_cvt_float_to_fp8(v / scale, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 e4m3_of8(const float (&v)[8], float scale) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        u[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] / scale, v[2 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
}

// kMode: 0 rotation alone, 1 append to an FP16 cache, 2 to an E4M3 cache.
// kVec: elements of a task's chunk, 8 or 1.
template <int kMode, int kLayout, int kVec>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(Job job) {
    // cosines and sines: [token of the CTA][R / 2], the eight pairs of rotating task k as four
    // float4s at k, rot + k, 2 rot + k, 3 rot + k (neighbouring threads read neighbouring words)
    extern __shared__ __align__(16) float2 turn[];
    pdl_launch_dependents();
    pdl_wait();  // everything read or written here may belong to the previous kernel
    const int half = job.r.R / 2;
    const int64_t t0 = (int64_t)blockIdx.x * job.tokens;
    const int nt = (int)(job.T - t0 < job.tokens ? job.T - t0 : job.tokens);
    const int rot_tasks = job.H * job.per_head, per_token = rot_tasks + job.copy_heads * job.per_copy;
    const int total = nt * per_token;

    struct Task {
        int token, head, at0, at1, pair;  // elements of the two chunks in the head (at1 < 0: one), first pair (-1: copy)
    };
    auto task_of = [&](int u) {
        Task k;
        k.token = 0;
        if (job.tokens > 1) {
            k.token = u / per_token;
            u -= k.token * per_token;
        }
        int i;
        if (kMode == 0 || u < rot_tasks) {
            k.head = job.head_shift >= 0 ? u >> job.head_shift : u / job.per_head;
            i = u - k.head * job.per_head;
        } else {
            u -= rot_tasks;
            k.head = u / job.per_copy;
            i = u - k.head * job.per_copy + job.rot;
            k.head += job.H;
        }
        const bool value = kMode != 0 && k.head >= job.H;
        if (!value && i < job.rot) {
            k.pair = i * kVec;
            // half: elements 8i .. and their partners; interleaved: 16-byte chunks i and rot + i
            k.at0 = kLayout == 0 || kVec == 8 ? k.pair : 2 * k.pair;
            k.at1 = kLayout == 0 || kVec == 8 ? k.pair + half : 2 * k.pair + 1;
        } else {
            k.pair = -1;
            k.at0 = (value ? 0 : job.r.R) + (i - job.rot) * 2 * kVec;
            k.at1 = k.at0 + kVec < job.D ? k.at0 + kVec : -1;
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
            if constexpr (kVec == 8) {
                w0[j] = *reinterpret_cast<const uint4 *>(row + k.at0);
                if (k.at1 >= 0) w1[j] = *reinterpret_cast<const uint4 *>(row + k.at1);
            } else {
                w0[j].x = row[k.at0];
                if (k.at1 >= 0) w1[j].x = row[k.at1];
            }
            sc[j] = 1.f;
            if (kMode == 2 && k.head >= job.Hq)
                sc[j] = __ldcg((k.head < job.H ? job.c.k_scale : job.c.v_scale) + kv_head(k));
        }
    };
    load(0);
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int token = i / half;
        const int pair = i - token * half;
        int at = pair;
        if constexpr (kVec == 8) {
            int task, quarter;  // of the pair's float4
            if (kLayout == 0) {
                task = pair >> 3, quarter = (pair & 7) >> 1;
            } else {
                const int chunk = pair >> 2, second = chunk >= job.rot;
                task = second ? chunk - job.rot : chunk, quarter = 2 * second + ((pair & 3) >> 1);
            }
            at = (quarter * job.rot + task) * 2 + (pair & 1);
        }
        turn[token * half + at] =
            sincos_at(__ldcg(job.r.positions + t0 + token), __ldcg(job.r.freqs + pair), job.r.magnitude);
    }
    // row of the tokens' entries in the pools' first head (or -1), in rows of D elements
    __shared__ int64_t entry[kMaxTokens];
    if (kMode != 0 && (int)threadIdx.x < nt) {
        const int64_t slot = __ldcg(job.slots + t0 + threadIdx.x);
        if (slot >= job.c.pages * job.c.page_size) atomicOr(job.status, kDevStatusCacheRange);
        const bool in = slot >= 0 && slot < job.c.pages * job.c.page_size;
        entry[threadIdx.x] = in ? (((slot >> job.page_shift) * job.c.kv_heads) << job.page_shift) + (slot & (job.c.page_size - 1)) : -1;
    }
    __syncthreads();
    auto finish = [&](const Task &k, const uint4 &c0, const uint4 &c1, float scale) {
        constexpr int n = kVec;
        float a[8], b[8];
        if constexpr (n == 8) {
            unpack8(c0, a);
            unpack8(c1, b);
        } else {
            a[0] = half_bits_to_float((uint16_t)c0.x), b[0] = half_bits_to_float((uint16_t)c1.x);
        }
        if (k.pair >= 0) {
            const float2 *cs = turn + k.token * half;
            if constexpr (n == 1) {
                const float2 f = cs[k.pair];
                const float p = a[0], q = b[0];
                a[0] = p * f.x - q * f.y;
                b[0] = q * f.x + p * f.y;
            } else {
                float2 f[8];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 v = reinterpret_cast<const float4 *>(cs)[i * job.rot + k.pair / 8];
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
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float p = a[2 * i], q = a[2 * i + 1], r = b[2 * i], t = b[2 * i + 1];
                        a[2 * i] = p * f[i].x - q * f[i].y;
                        a[2 * i + 1] = q * f[i].x + p * f[i].y;
                        b[2 * i] = r * f[i + 4].x - t * f[i + 4].y;
                        b[2 * i + 1] = t * f[i + 4].x + r * f[i + 4].y;
                    }
                }
            }
        }
        auto put16 = [&](uint16_t *row) {
            if constexpr (n == 8) {
                *reinterpret_cast<uint4 *>(row + k.at0) = pack8(a);
                if (k.at1 >= 0) *reinterpret_cast<uint4 *>(row + k.at1) = pack8(b);
            } else {
                row[k.at0] = float_to_half_bits(a[0]);
                if (k.at1 >= 0) row[k.at1] = float_to_half_bits(b[0]);
            }
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
                    if constexpr (n == 8) {
                        *reinterpret_cast<uint2 *>(row + k.at0) = e4m3_of8(a, scale);
                        if (k.at1 >= 0) *reinterpret_cast<uint2 *>(row + k.at1) = e4m3_of8(b, scale);
                    } else {
                        row[k.at0] = e4m3_of(a[0], scale);
                        if (k.at1 >= 0) row[k.at1] = e4m3_of(b[0], scale);
                    }
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
    const bool vec = R % 16 == 0;
    const int v = vec ? 8 : 1;
    job.rot = R / 2 / v;
    // in place, what is not rotated already is where it belongs
    const bool in_place = kMode == 0 && job.x == job.out;
    job.per_head = job.rot + (in_place ? 0 : (D - R + 2 * v - 1) / (2 * v));
    job.per_copy = (D + 2 * v - 1) / (2 * v);
    const int64_t per_token = (int64_t)job.H * job.per_head + (int64_t)job.copy_heads * job.per_copy;
    if (per_token == 0) return cudaSuccess;
    // several small tokens per CTA, as long as every SM still gets four CTAs
    int64_t tokens = 256 / per_token;
    const int64_t spread = job.T / (4 * (int64_t)dev.sm_count);
    tokens = tokens < spread ? tokens : spread;
    tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
    job.tokens = (int)tokens;
    // Few tokens: every task its own thread (32 tokens of 448 tasks: 3.3 us with 512 threads, 4.9
    // with 128).  Many: four tasks per thread keep more loads in flight per CTA and fewer warps at
    // its barrier (8191 tokens of 384 tasks: 41 us with 128 threads, 50 with 256).
    int64_t threads = job.T < 2 * (int64_t)dev.sm_count ? per_token * tokens : 128;
    threads = threads > kMaxThreads ? kMaxThreads : threads < 64 ? 64 : (threads + 31) / 32 * 32;
    job.head_shift = -1;
    for (int i = 0; i < 16; i++)
        if (job.per_head == 1 << i) job.head_shift = i;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((job.T + tokens - 1) / tokens));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)tokens * (size_t)(R / 2) * sizeof(float2);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (vec)
        return cudaLaunchKernelEx(&cfg, job.r.layout == 0 ? rope_kernel<kMode, 0, 8> : rope_kernel<kMode, 1, 8>, job);
    return cudaLaunchKernelEx(&cfg, job.r.layout == 0 ? rope_kernel<kMode, 0, 1> : rope_kernel<kMode, 1, 1>, job);
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

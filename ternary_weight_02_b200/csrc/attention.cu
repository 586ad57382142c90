// attention.cu -- attention of one new token per sequence over a paged key/value cache.
//
// out = sum_j p_j v_j, p = softmax_j(scale * q . k_j), in one pass over the cache: a running
// maximum m and sum l of e^(z - m), the weighted sum of the values rescaled whenever m grows.
// One CTA per (sequence, query head), one warp per key in turn, the warps joined at the end.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace bonsai {
namespace {

constexpr int kWarps = 4;

template <int D, int kType>
__device__ __forceinline__ void load_row(const void *pool, int64_t row, int lane, float (&v)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; i++) {
        if (kType == 0)
            v[i] = half_bits_to_float(static_cast<const uint16_t *>(pool)[row * D + i * 32 + lane]);
        else
            v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(
                static_cast<const __nv_fp8_storage_t *>(pool)[row * D + i * 32 + lane], __NV_E4M3)));
    }
}

template <int D, int kType>
__global__ void __launch_bounds__(32 * kWarps) attention_kernel(const uint16_t *q, KvCache c, const int32_t *table,
                                                                const int32_t *lengths, uint16_t *out, float *lse,
                                                                int64_t Hq, int64_t ld_q, int64_t ld_out, int64_t width,
                                                                int64_t window, float scale, unsigned int *status) {
    const int64_t b = blockIdx.x / Hq, h = blockIdx.x % Hq, hk = h / (Hq / c.kv_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cap = width * c.page_size, given = lengths[b];
    bool bad = given < 0 || given > cap;
    const int64_t len = given < 0 ? 0 : given > cap ? cap : given;
    const int64_t first = window > 0 && len > window ? len - window : 0;
    const float ks = kType ? c.k_scale[hk] : 1.f, vs = kType ? c.v_scale[hk] : 1.f;
    float qv[D / 32], acc[D / 32] = {}, m = -INFINITY, l = 0.f;
    load_row<D, 0>(q + b * ld_q + h * D, 0, lane, qv);
    for (int64_t j = first + warp; j < len; j += kWarps) {
        const int64_t page = table[b * width + j / c.page_size];
        if (page < 0 || page >= c.pages) {
            bad = true;
            continue;
        }
        const int64_t row = (page * c.kv_heads + hk) * c.page_size + j % c.page_size;
        float k[D / 32], v[D / 32];
        load_row<D, kType>(c.k, row, lane, k);
        load_row<D, kType>(c.v, row, lane, v);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; i++) z += qv[i] * k[i];
        z = warp_sum(z) * scale * ks;
        const float mn = fmaxf(m, z), f = m == mn ? 1.f : expf(m - mn), p = expf(z - mn);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < D / 32; i++) acc[i] = acc[i] * f + p * v[i];
        m = mn;
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < D / 32; i++) so[warp][i * 32 + lane] = acc[i];
    bad = __syncthreads_or(bad);
    float mt = -INFINITY, lt = 0.f;
    for (int w = 0; w < kWarps; w++) mt = fmaxf(mt, sm[w]);
    for (int w = 0; w < kWarps; w++) lt += sl[w] == 0.f ? 0.f : sl[w] * expf(sm[w] - mt);
    const float nan = __int_as_float(0x7fc00000);
    for (int i = threadIdx.x; i < D; i += 32 * kWarps) {
        float o = 0.f;
        for (int w = 0; w < kWarps; w++)
            if (sl[w] != 0.f) o += so[w][i] * expf(sm[w] - mt);
        o = len == first ? 0.f : o / lt * vs;
        out[b * ld_out + h * D + i] = float_to_half_bits(bad ? nan : o);
    }
    if (threadIdx.x == 0) {
        if (lse) lse[b * Hq + h] = bad ? nan : len == first ? -INFINITY : mt + logf(lt);
        if (bad) atomicOr(status, kDevStatusCacheRange);
    }
}

}  // namespace

size_t attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, const DeviceInfo &dev) {
    (void)B, (void)Hq, (void)Hkv, (void)D, (void)dev;
    return 0;
}

cudaError_t launch_paged_attention(const uint16_t *q, const KvCache &c, const int32_t *table, const int32_t *lengths,
                                   uint16_t *out, float *lse, int64_t B, int64_t Hq, int64_t ld_q, int64_t ld_out,
                                   int64_t width, int64_t window, float scale, const Workspace &ws, cudaStream_t s,
                                   const DeviceInfo &dev) {
    (void)dev;
    unsigned int *status = reinterpret_cast<unsigned int *>(ws.zeroed) + kCtlStatus;
    auto go = [&](auto kern) {
        kern<<<(unsigned)(B * Hq), 32 * kWarps, 0, s>>>(q, c, table, lengths, out, lse, Hq, ld_q, ld_out, width, window,
                                                       scale, status);
        return cudaGetLastError();
    };
    if (c.type == 0)
        return c.head_dim == 64    ? go(attention_kernel<64, 0>)
               : c.head_dim == 128 ? go(attention_kernel<128, 0>)
                                   : go(attention_kernel<256, 0>);
    return c.head_dim == 64    ? go(attention_kernel<64, 1>)
           : c.head_dim == 128 ? go(attention_kernel<128, 1>)
                               : go(attention_kernel<256, 1>);
}

}  // namespace bonsai

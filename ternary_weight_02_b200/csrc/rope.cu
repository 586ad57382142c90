// rope.cu -- rotary positions, alone and with the append of keys and values to a paged cache.
//
// A pair (a, b) of a head at position p turns by the angle p * f of its frequency f:
// (a, b) -> magnitude * (a cos - b sin, b cos + a sin).  The angle is a product of up to
// 10^6 positions and a frequency: in FP32 its absolute error would pass the FP16 rounding
// of the result from a few thousand positions on, so it is formed in FP64, counted in turns
// and reduced to [-1/2, 1/2] there; sine and cosine of the rest are FP32.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace bonsai {
namespace {

__device__ __forceinline__ void sincos_at(int pos, double freq, float magnitude, float *c, float *s) {
    double turns = (double)pos * freq * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float sn, cs;
    sincospif(2.f * (float)turns, &sn, &cs);
    *c = magnitude * cs;
    *s = magnitude * sn;
}

// Element i of a head rotated (i < R), from the pair it belongs to.
__device__ __forceinline__ float rotated(const uint16_t *head, int i, int R, int layout, int pos, const double *freqs,
                                         float magnitude) {
    const int pair = layout == 0 ? (i < R / 2 ? i : i - R / 2) : i >> 1;
    const int ia = layout == 0 ? pair : 2 * pair, ib = layout == 0 ? pair + R / 2 : 2 * pair + 1;
    float c, s;
    sincos_at(pos, freqs[pair], magnitude, &c, &s);
    const float a = half_bits_to_float(head[ia]), b = half_bits_to_float(head[ib]);
    return i == ia ? a * c - b * s : b * c + a * s;
}

// One CTA per token and head; the head's values are all read before any is written (x may be out).
__global__ void rope_kernel(const uint16_t *x, uint16_t *out, RopeArgs r, int64_t H, int64_t D, int64_t ld_x,
                            int64_t ld_out) {
    const int64_t t = blockIdx.x / H, h = blockIdx.x % H;
    const uint16_t *head = x + t * ld_x + h * D;
    const int pos = r.positions[t], i = threadIdx.x;
    float v = 0.f;
    if (i < D) v = i < r.R ? rotated(head, i, r.R, r.layout, pos, r.freqs, r.magnitude) : half_bits_to_float(head[i]);
    __syncthreads();
    if (i < D) out[t * ld_out + h * D + i] = float_to_half_bits(v);
}

__global__ void rope_append_kernel(const uint16_t *qkv, uint16_t *q_out, KvCache c, RopeArgs r, const int64_t *slots,
                                   int64_t Hq, int64_t ld_qkv, int64_t ld_q, unsigned int *status) {
    const int64_t Hkv = c.kv_heads, D = c.head_dim, H = Hq + 2 * Hkv;
    const int64_t t = blockIdx.x / H, h = blockIdx.x % H;
    const uint16_t *head = qkv + t * ld_qkv + h * D;
    const int pos = r.positions[t], i = threadIdx.x;
    const bool turn = h < Hq + Hkv && i < r.R;
    const float v = turn ? rotated(head, i, r.R, r.layout, pos, r.freqs, r.magnitude) : half_bits_to_float(head[i]);
    __syncthreads();
    if (h < Hq) {
        q_out[t * ld_q + h * D + i] = float_to_half_bits(v);
        return;
    }
    const int64_t slot = slots[t];
    if (slot < 0) return;
    if (slot >= c.pages * c.page_size) {
        if (i == 0) atomicOr(status, kDevStatusCacheRange);
        return;
    }
    const bool is_k = h < Hq + Hkv;
    const int64_t hk = is_k ? h - Hq : h - Hq - Hkv;
    const int64_t at = ((slot / c.page_size * Hkv + hk) * c.page_size + slot % c.page_size) * D + i;
    void *pool = is_k ? c.k : c.v;
    if (c.type == 0)
        static_cast<uint16_t *>(pool)[at] = float_to_half_bits(v);
    else
        static_cast<__nv_fp8_storage_t *>(pool)[at] =
            __nv_cvt_float_to_fp8(v / (is_k ? c.k_scale : c.v_scale)[hk], __NV_SATFINITE, __NV_E4M3);
}

}  // namespace

cudaError_t launch_rope(const uint16_t *x, uint16_t *out, const RopeArgs &r, int64_t T, int64_t H, int64_t D,
                        int64_t ld_x, int64_t ld_out, cudaStream_t s, const DeviceInfo &dev) {
    (void)dev;
    rope_kernel<<<(unsigned)(T * H), (unsigned)((D + 31) / 32 * 32), 0, s>>>(x, out, r, H, D, ld_x, ld_out);
    return cudaGetLastError();
}

cudaError_t launch_rope_append(const uint16_t *qkv, uint16_t *q_out, const KvCache &c, const RopeArgs &r,
                               const int64_t *slots, int64_t T, int64_t Hq, int64_t ld_qkv, int64_t ld_q,
                               const Workspace &ws, cudaStream_t s, const DeviceInfo &dev) {
    (void)dev;
    unsigned int *status = reinterpret_cast<unsigned int *>(ws.zeroed) + kCtlStatus;
    rope_append_kernel<<<(unsigned)(T * (Hq + 2 * c.kv_heads)), (unsigned)c.head_dim, 0, s>>>(qkv, q_out, c, r, slots,
                                                                                           Hq, ld_qkv, ld_q, status);
    return cudaGetLastError();
}

}  // namespace bonsai

// attention.cu -- attention of one new token per sequence over a paged key/value cache.
//
// out = sum_j p_j v_j, p = softmax_j(scale * q . k_j), in one pass over the cache: a running
// maximum m and sum l of 2^(z - m) (z in base-2 units), the weighted sum of the values
// rescaled whenever m grows; parts over different keys join by the same rule.
//
// HBM-bound: each key and value is read once and meets the G = Hq / Hkv query heads that share
// it, 4 G flops per FP16 element pair, far below the tensor cores' rate.  So the design serves
// the copies:
//
// * Units of work are tiles of 64, 128 or 256 keys of one (sequence, key/value head, tile of 8 NT query
//   heads).  All units of the call lie in one list, sequence by sequence, and each CTA of a
//   grid that is resident at once takes an equal run of it: a ragged batch loads every SM
//   alike, one long sequence spreads over all of them, and the host needs no lengths (a
//   captured call follows them).  Every CTA finds its run from a scan of the lengths.
// * A producer warp walks the run's tiles, across sequences, and keeps a ring of kStages tiles
//   in flight by TMA: one box per page and pool, 128-byte (64-byte for 64-byte rows) swizzle.
//   Page numbers are read 32 at a time, checked, and never followed when out of range.  Three
//   CTAs of two 32 KB stages per SM beat two of three (64 ragged sequences 82 against 86 us):
//   the consumers' latency, not the bytes in flight, is what more of them hides.
// * kWarps consumer warps take 16 keys of each tile (two blocks of 16 where a row has 128 bytes
//   or fewer: E4M3 ragged 96 against 103 us; four of 64 bytes; one again where 16 query heads of
//   128 fill the registers, so that two CTAs fit: 16 heads per key head, E4M3, 68 against 74 us):
//   S^T = K Q^T as m16n8k16 MMAs with the keys as rows, so that 8 query heads fill the columns and no row is wasted on padding; the
//   probabilities, times 2^14, are rounded to FP16 (2^-11 of each, the size of the output's own
//   rounding, down to 2^-28 of the largest), transposed by movmatrix into the B operand of O^T += V^T P^T.  Each warp keeps
//   its own m, l and O; they meet once per piece of a run.
// * E4M3 entries become FP16 in registers (exactly); the per-head scales go into the score
//   scale and the output.  The contraction indices are taken in the order in which the bytes
//   arrive, Q being loaded in the same order.
// * A (sequence, head) that spans CTAs leaves partial (m, l, O) in the workspace; the CTA that
//   arrives last adds them up in run order (repeatable), so no CTA waits for another.
//
// Waits are bounded.  A consumer warp whose copy never lands gives up: its pieces become NaN, the
// status bit is set, the joins run as ever, so that their counters end at zero.  The producer, whose
// stages are then never freed, gives up too; and it leaves only when every copy that it started has
// landed, since a copy must not outlive its CTA's shared memory.
//
// Keys outside the sequence's window get a score of -infinity, and their values are masked to
// zero in the MMA operand (a NaN there times a zero probability would be a NaN).

#include "common.cuh"
#include "internal.h"
#include "tma.cuh"

namespace bonsai {
namespace {

constexpr int kWarps = 4;  // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
// Parts of an item that one CTA adds up at once; more go in groups.  (131072 keys, 8 heads, 56
// parts: 87.9 us in groups, 92.8 us at once; 1024 keys, 16 parts: 10.4 against 9.0 us.)
constexpr int kFlatParts = 20;
// Probabilities, their sum l and the weighted values are held times 2^kLift: a probability of the
// maximum is 2^14 in FP16 (whose largest value is almost 2^16), and one that falls below FP16's
// normal range is under 2^-28 of the maximum, where its rounding of 2^-39 is lost on no context
// (unlifted, 2^-25 for each of 131072 keys could add up to 2^-8).
// The lift multiplies 2^(z - m), whose argument is formed first: with the lift in the exponent as
// 2^(z - (m - 14)), m - 14 is no longer m less 14 from |m| = 2^25 on (m = 4e7: 2^16, an infinity in
// FP16).  131072 keys 87.6 us, 87.5 with the lift in the exponent.
constexpr float kLift = 14.f, kLifted = 16384.f;

template <int D, int kType, int NT>
struct Cfg {
    static constexpr int kRowBytes = kType == 0 ? 2 * D : D;
    static constexpr int kInner = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a box row
    // 16-key blocks of a warp in a tile: more for short rows, whose keys cost more than their bytes
    static constexpr int kBlk = kRowBytes == 64 && NT == 1 ? 4 : kRowBytes <= 128 && NT * D <= 128 ? 2 : 1;
    static constexpr int kTile = 16 * kWarps * kBlk;                  // keys of a tile
    // CTAs per SM that the registers leave room for (the ring takes the rest of the shared memory)
    static constexpr int kCtas = D == 256 ? (NT == 2 || kType == 0 ? 1 : 2)
                                 : NT == 2 && D == 128 ? 2 : NT == 1 && D == 64 && kType == 0 ? 4 : 3;
    static constexpr int kPoolBytes = kTile * kRowBytes;              // one pool's part of a stage
    static constexpr int kStageBytes = 2 * kPoolBytes;
    static constexpr int kStages = kStageBytes > 32768 ? 3 : kStageBytes > 16384 ? 2 : 4;
};

struct Layout {
    int join, ml, bars, total;  // byte offsets after the ring
};
template <int D, int kType, int NT>
constexpr Layout layout() {
    using C = Cfg<D, kType, NT>;
    Layout l{};
    l.join = C::kStages * C::kStageBytes;            // 2 x [NT][D / 16][32] float4
    l.ml = l.join + 2 * 8 * NT * D * 4;              // m and l: [2][kWarps][8 NT]
    l.bars = l.ml + 2 * kWarps * 8 * NT * 4;         // full, empty, bad[stage]
    l.total = l.bars + C::kStages * (8 + 8 + 4) + 1024 + 64;
    return l;
}

struct Params {
    const uint16_t *q;
    const float *k_scale, *v_scale;
    const int32_t *table, *lengths;
    uint16_t *out;
    float *lse, *partials;
    unsigned int *counters, *status;
    int64_t ld_q, ld_out, width, window, cap;  // cap: width * page_size
    int B, Hq, Hkv, G, GT;                      // GT: query tiles of a key/value head
    int pages, page_shift;
    float scale;
    uint32_t wait_limit;  // polls of the ring's waits
    bool force_timeouts;  // test hook: the consumers wait for a copy that nobody makes
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(saddr(dst)), "l"(map), "r"(saddr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 values as FP16, exactly: bytes 0, 1 in lo, bytes 2, 3 in hi.
__device__ __forceinline__ void e4m3x4_to_half(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
// 2^x, x <= 0 or -infinity: relative error 2^-22
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Loads through L2 that are issued where they stand: several in flight before the first use.
__device__ __forceinline__ float2 load_now(const float2 *p) {
    float2 v;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_now(const float4 *p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
// 2^(m - top), 0 for a part without keys (m = -infinity; top may be too)
__device__ __forceinline__ float weight_of(float m, float top) { return m == -INFINITY ? 0.f : exp2_fast(m - top); }

// a / b for a >= 0, b > 0: 32-bit where both fit (the 64-bit division is a long routine)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Keys of sequence b that take part, [first, len), and the tiles they lie in.
struct Span {
    int64_t first, len;
    int tile0, tiles;
    bool bad;
};
template <int kTile>
__device__ __forceinline__ Span span_of(const Params &p, int given) {
    Span s;
    s.bad = given < 0 || given > p.cap;
    s.len = given < 0 ? 0 : given > p.cap ? p.cap : given;
    s.first = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
    s.tile0 = (int)(s.first / kTile);
    const int n = (int)((s.len + kTile - 1) / kTile) - s.tile0;
    s.tiles = n > 0 ? n : 1;  // an empty sequence has one tile without keys
    return s;
}

// A walk over a run of units: item by item, an item being (sequence, head, query tile).
template <int kTile>
struct Walk {
    int b, hg, t;       // sequence, (head, query tile) in it, tile of the item
    int64_t left;       // units left of the run
    int next_len;
    Span s;
    __device__ __forceinline__ void enter(const Params &p) {
        s = span_of<kTile>(p, next_len);
        next_len = b + 1 < p.B ? __ldcg(p.lengths + b + 1) : 0;
    }
    __device__ __forceinline__ void start(const Params &p, int b0, int len0, int64_t off, int64_t units) {
        b = b0;
        left = units;
        next_len = len0;
        enter(p);
        hg = (int)divide(off, s.tiles);
        t = (int)(off - (int64_t)hg * s.tiles);
    }
    // the piece of the current item in this run: tiles [t, end)
    __device__ __forceinline__ int end() const { return (int64_t)(s.tiles - t) < left ? s.tiles : t + (int)left; }
    __device__ __forceinline__ void next(const Params &p, int end) {
        left -= end - t;
        t = 0;
        if (++hg == p.Hkv * p.GT) {
            hg = 0;
            if (++b == p.B) left = 0;  // (the lengths changed under the call: stop at the last sequence)
            if (left > 0) enter(p);
        }
    }
};

template <int D, int kType, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, kType, NT>::kCtas) attention_kernel(const __grid_constant__ CUtensorMap k_map,
                                                             const __grid_constant__ CUtensorMap v_map, Params p) {
    using C = Cfg<D, kType, NT>;
    constexpr Layout L = layout<D, kType, NT>();
    constexpr int kTile = C::kTile, kBlk = C::kBlk;
    constexpr int kQ = 8 * NT;                 // query heads of an item
    constexpr int kSlot = kQ * (D + 2);        // floats of a partial result: O, then m, l
    constexpr bool kQRegs = NT * D <= 256;     // Q fragments in registers, else re-read per tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    float4 *join = reinterpret_cast<float4 *>(smem + L.join);
    float *sm = reinterpret_cast<float *>(smem + L.ml), *sl = sm + kWarps * kQ;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L.bars), *empty = full + C::kStages;
    volatile int *bad_page = reinterpret_cast<int *>(empty + C::kStages);
    __shared__ int64_t scan_warp[kWarps + 1], start_off;
    __shared__ int start_b, start_len, last_flag;
    __shared__ uint64_t never;  // a barrier that nobody arrives on

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; i++) mbar_init(full + i, 1), mbar_init(empty + i, kWarps);
        mbar_init(&never, 1);
        mbar_init_fence();
    }
    pdl_launch_dependents();
    pdl_wait();  // everything read or written here may belong to the previous kernel

    // ---- this CTA's run of units: thread i sums a stretch of the sequences' tiles
    const int per = (p.B + kThreads - 1) / kThreads;
    const int bs = tid * per < p.B ? tid * per : p.B, be = bs + per < p.B ? bs + per : p.B;
    int64_t mine = 0;
    int len = 0;  // the stretch's last length
    for (int b = bs; b < be; b++) mine += span_of<kTile>(p, len = __ldcg(p.lengths + b)).tiles;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan_warp[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, tiles = 0;
    for (int w = 0; w <= kWarps; w++) {
        if (w < warp) before += scan_warp[w];
        tiles += scan_warp[w];
    }
    const int64_t HG = (int64_t)p.Hkv * p.GT, W = tiles * HG;
    const int64_t nc = W < (int64_t)gridDim.x ? W : (int64_t)gridDim.x;  // CTAs with work
    const int64_t cta = blockIdx.x;
    if (cta >= nc) return;
    const int64_t w0 = divide(W * cta, nc), w1 = divide(W * (cta + 1), nc);
    if (w0 >= before * HG && w0 < (before + mine) * HG) {  // one thread: the run starts in its stretch
        int64_t at = before * HG;
        int b = bs;
        for (; be - b > 1; b++) {  // (the last is the one whose length is at hand)
            const int v = __ldcg(p.lengths + b);
            const int64_t n = span_of<kTile>(p, v).tiles * HG;
            if (w0 < at + n) {
                len = v;
                break;
            }
            at += n;
        }
        start_b = b;
        start_len = len;
        start_off = w0 - at;
    }
    __syncthreads();
    Walk<kTile> walk;
    walk.start(p, start_b, start_len, start_off, w1 - w0);
    const int slab = 1 << p.page_shift < kTile ? 1 << p.page_shift : kTile;  // keys of a box

    if (warp == kWarps) {
        // ---------------------------------------------------------------- producer
        const int slabs = kTile / slab;  // boxes of a tile and pool
        int st = 0, issued = 0;
        uint32_t phase = 1;  // the first pass over the ring finds every stage empty
        // every stage's last copy has landed (the consumers may have given up on it)
        auto drain = [&]() {
            for (int i = issued < C::kStages ? 0 : issued - C::kStages; i < issued; i++)
                mbar_wait(full + i % C::kStages, (uint32_t)(i / C::kStages) & 1u);
        };
        while (walk.left > 0) {
            const int end = walk.end();
            const int hk = walk.hg / p.GT;
            const int32_t *row = p.table + (int64_t)walk.b * p.width;
            const Span s = walk.s;
            // page of the slab n of this piece: read 32 at a time, the next 32 ahead
            const int64_t key0 = (int64_t)(s.tile0 + walk.t) * kTile;
            const int total = (end - walk.t) * slabs;
            auto page_of = [&](int n) -> int {
                const int64_t key = key0 + (int64_t)n * slab;
                if (n >= total || key >= s.len || key + slab <= s.first) return -2;  // no key in use
                const int page = __ldcg(row + (key >> p.page_shift));
                return page >= 0 && page < p.pages ? page : -1;
            };
            int ids = page_of(lane), ahead = page_of(32 + lane);
            for (int n = 0; n < total; n += slabs) {
                if (n > 0 && (n & 31) == 0) {
                    ids = ahead;
                    ahead = page_of(n + 32 + lane);
                }
                if (!__all_sync(0xffffffffu, mbar_wait(empty + st, phase, p.wait_limit))) {  // the consumers gave up
                    drain();
                    return;
                }
                int valid = 0, bad = 0;
                for (int i = 0; i < slabs; i++) {
                    const int id = __shfl_sync(0xffffffffu, ids, (n + i) & 31);
                    valid += id >= 0;
                    bad |= id == -1;
                }
                if (lane == 0) {
                    bad_page[st] = bad;
                    if (bad) atomicOr(p.status, kDevStatusCacheRange);
                    mbar_arrive_expect_tx(full + st, (uint32_t)(valid * 2 * slab * C::kRowBytes));
                }
                __syncwarp();
                uint8_t *dst = smem + st * C::kStageBytes;
                for (int i = 0; i < slabs; i++) {
                    const int id = __shfl_sync(0xffffffffu, ids, (n + i) & 31);
                    if (id < 0 || lane != 0) continue;
                    const int place = (int)((key0 + (int64_t)(n + i) * slab) & ((1 << p.page_shift) - 1));
                    const int off = i * slab * C::kRowBytes;
                    tma_load_4d(dst + off, &k_map, full + st, 0, place, 0, id * p.Hkv + hk);
                    tma_load_4d(dst + C::kPoolBytes + off, &v_map, full + st, 0, place, 0, id * p.Hkv + hk);
                }
                issued++;
                if (++st == C::kStages) st = 0, phase ^= 1;
            }
            walk.next(p, end);
        }
        drain();
        return;
    }

    // -------------------------------------------------------------------- consumers
    // ldmatrix addresses: matrix mi of four, row r8 of its eight.  A row's 16-byte chunk c lies in
    // 128-byte block c / 8 (each `slab` rows tall), at place c % 8 xored with the row's swizzle
    // bits; as nothing else sets those address bits, the xor takes the whole address.
    const int mi = lane >> 3, r8 = lane & 7;
    const int key_k = r8 + (mi & 1) * 8, chunk_k = mi >> 1;
    const int key_v = r8 + (kType == 0 ? (mi >> 1) * 8 : (mi & 1) * 8), chunk_v = kType == 0 ? (mi & 1) : (mi >> 1);
    // block j of this warp: keys 64 j + 16 warp .. + 15 of the tile, within one slab
    auto lane_off = [&](int j, int key, int chunk) -> uint32_t {
        const int first = 16 * (j * kWarps + warp), row = (first & (slab - 1)) + key;
        const int x = C::kInner == 128 ? row & 7 : (row >> 1) & 3;
        return (uint32_t)(first / slab * slab * C::kRowBytes + row * C::kInner + ((chunk ^ x) << 4));
    };
    uint32_t off_k[kBlk], off_v[kBlk];
#pragma unroll
    for (int j = 0; j < kBlk; j++) {
        off_k[j] = lane_off(j, key_k, chunk_k);
        off_v[j] = C::kPoolBytes + lane_off(j, key_v, chunk_v);
    }
    const uint32_t block_bytes = slab * C::kInner;
    auto chunk_addr = [&](uint32_t base, int c) -> uint32_t {  // c even
        constexpr int kChunks = C::kInner / 16;
        return (base ^ ((c & (kChunks - 1)) << 4)) + (c / kChunks) * block_bytes;
    };
    bool alive = true;
    int st = 0;
    uint32_t phase = 0;
    while (walk.left > 0) {
        const int end = walk.end();
        const Span s = walk.s;
        const int b = walk.b, hk = walk.hg / p.GT, q0 = (walk.hg - hk * p.GT) * kQ;  // first query of the tile in the group
        const int64_t head0 = (int64_t)hk * p.G + q0;
        const int nq = p.G - q0 < kQ ? p.G - q0 : kQ;
        const float to2 = p.scale * 1.44269504088896340736f * (kType ? __ldcg(p.k_scale + hk) : 1.f);

        // Q as B operands: query gid of each n-tile, contraction pairs in the K operand's order
        uint32_t qf[kQRegs ? NT : 1][kQRegs ? D / 16 : 1][2];
        auto load_q = [&](int nt, int ks, uint32_t &b0, uint32_t &b1) {
            const int qi = nt * 8 + gid;
            b0 = b1 = 0;
            if (qi >= nq) return;
            const uint16_t *row = p.q + (int64_t)b * p.ld_q + (head0 + qi) * D + 16 * ks;
            if (kType == 0) {
                b0 = *reinterpret_cast<const uint32_t *>(row + 2 * tig);
                b1 = *reinterpret_cast<const uint32_t *>(row + 8 + 2 * tig);
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(row + 4 * tig);
                b0 = v.x, b1 = v.y;
            }
        };
        if constexpr (kQRegs) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++) load_q(nt, ks, qf[nt][ks][0], qf[nt][ks][1]);
        }
        float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; i++) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
        }
        bool nan = s.bad;
        for (int t = walk.t; t < end; t++) {
            if (alive && !mbar_wait(p.force_timeouts ? &never : full + st, p.force_timeouts ? 0 : phase, p.wait_limit)) {
                alive = false;
                if (lane == 0) atomicOr(p.status, kDevStatusAttentionTimeout);
            }
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) {
                nan = true;
                continue;
            }
            nan = nan || bad_page[st] != 0;
            const uint32_t stage = saddr(smem + st * C::kStageBytes);
            const int64_t key0 = (int64_t)(s.tile0 + t) * kTile + 16 * warp;
            constexpr int kStep = 16 * kWarps;  // keys between a warp's blocks
            if (key0 < s.len && key0 + (kBlk - 1) * kStep + 16 > s.first) {  // (uniform in the warp) it has keys here
                float z[kBlk][NT][4];
#pragma unroll
                for (int j = 0; j < kBlk; j++)
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) z[j][nt][0] = z[j][nt][1] = z[j][nt][2] = z[j][nt][3] = 0.f;
                auto score = [&](int j, int ks, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        if constexpr (kQRegs) {
                            mma16816(z[j][nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
                        } else {
                            uint32_t b0, b1;
                            load_q(nt, ks, b0, b1);
                            mma16816(z[j][nt], a0, a1, a2, a3, b0, b1);
                        }
                    }
                };
                if (kType == 0) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
                        for (int j = 0; j < kBlk; j++) {
                            uint32_t a[4];
                            ldmatrix4(a, chunk_addr(stage + off_k[j], 2 * ks));
                            score(j, ks, a[0], a[1], a[2], a[3]);
                        }
                } else {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ks += 2)  // 16-byte chunks ks, ks + 1 of rows gid, gid + 8
#pragma unroll
                        for (int j = 0; j < kBlk; j++) {
                            uint32_t a[4];
                            ldmatrix4(a, chunk_addr(stage + off_k[j], ks));
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_half(a[2 * i], a0, a2);
                                e4m3x4_to_half(a[2 * i + 1], a1, a3);
                                score(j, ks + i, a0, a1, a2, a3);
                            }
                        }
                }
                // keys gid and gid + 8 of a block's scores; keys 2 tig (+ 1, + 8, + 9) of its values
                const bool edge = key0 < s.first || key0 + (kBlk - 1) * kStep + 16 > s.len;
                uint32_t vm[kBlk][2];
#pragma unroll
                for (int j = 0; j < kBlk; j++) vm[j][0] = vm[j][1] = 0xffffffffu;
#pragma unroll
                for (int j = 0; j < kBlk; j++)
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        // (rounded here: fused into the differences below, z - m of the largest would be the
                        // rounding of the product, far from 0 for large scores)
                        for (int e = 0; e < 4; e++) z[j][nt][e] = __fmul_rn(z[j][nt][e], to2);
                if (edge) {
#pragma unroll
                    for (int j = 0; j < kBlk; j++) {
                        const int64_t kj = key0 + j * kStep;
                        auto in = [&](int i) { return kj + i >= s.first && kj + i < s.len; };
                        const bool in0 = in(gid), in1 = in(gid + 8);
                        vm[j][0] = (in(2 * tig) ? 0xffffu : 0u) | (in(2 * tig + 1) ? 0xffff0000u : 0u);
                        vm[j][1] = (in(2 * tig + 8) ? 0xffffu : 0u) | (in(2 * tig + 9) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if (!(e < 2 ? in0 : in1)) z[j][nt][e] = -INFINITY;
                    }
                }
                uint32_t pb[kBlk][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float top[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        float v = fmaxf(z[0][nt][e], z[0][nt][e + 2]);
#pragma unroll
                        for (int j = 1; j < kBlk; j++) v = fmaxf(v, fmaxf(z[j][nt][e], z[j][nt][e + 2]));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        top[e] = fmaxf(m[nt][e], v);
                    }
                    if (__any_sync(0xffffffffu, top[0] != m[nt][0] || top[1] != m[nt][1])) {
                        const float f0 = weight_of(m[nt][0], top[0]), f1 = weight_of(m[nt][1], top[1]);
                        m[nt][0] = top[0], m[nt][1] = top[1];
                        l[nt][0] *= f0, l[nt][1] *= f1;
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            o[nt][i][0] *= f0, o[nt][i][1] *= f1;
                            o[nt][i][2] *= f0, o[nt][i][3] *= f1;
                        }
                    }
                    // (a maximum of -infinity, every score being one: 2^(-inf - 0) = 0)
                    const float s0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
                    const float s1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                    for (int j = 0; j < kBlk; j++) {
                        auto lifted = [](float z, float s) { return kLifted * exp2_fast(__fsub_rn(z, s)); };
                        const float p0 = lifted(z[j][nt][0], s0), p1 = lifted(z[j][nt][1], s1);
                        const float p2 = lifted(z[j][nt][2], s0), p3 = lifted(z[j][nt][3], s1);
                        l[nt][0] += p0 + p2;
                        l[nt][1] += p1 + p3;
                        const __half2 h01 = __floats2half2_rn(p0, p1), h23 = __floats2half2_rn(p2, p3);
                        pb[j][nt][0] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h01));
                        pb[j][nt][1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h23));
                    }
                }
                auto weigh = [&](int j, int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                    if (edge) a0 &= vm[j][0], a1 &= vm[j][0], a2 &= vm[j][1], a3 &= vm[j][1];
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) mma16816(o[nt][i], a0, a1, a2, a3, pb[j][nt][0], pb[j][nt][1]);
                };
                if (kType == 0) {
#pragma unroll
                    for (int j = 0; j < kBlk; j++)
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            uint32_t a[4];
                            ldmatrix4_trans(a, chunk_addr(stage + off_v[j], 2 * i));
                            weigh(j, i, a[0], a[1], a[2], a[3]);
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < kBlk; j++)
#pragma unroll
                        for (int i = 0; i < D / 16; i += 2) {
                            uint32_t a[4];
                            ldmatrix4_trans(a, chunk_addr(stage + off_v[j], i));
#pragma unroll
                            for (int u = 0; u < 2; u++) {  // bytes (0, 2): dimension 2 gid, (1, 3): 2 gid + 1
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_half(__byte_perm(a[2 * u], 0, 0x3120), a0, a1);
                                e4m3x4_to_half(__byte_perm(a[2 * u + 1], 0, 0x3120), a2, a3);
                                weigh(j, i + u, a0, a1, a2, a3);
                            }
                        }
                }
            }
            // this warp's reads of the stage come before the copies that refill it
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
            if (++st == C::kStages) st = 0, phase ^= 1;
        }

        // ---- join the warps: m and l of every warp, then O scaled to the common maximum
        consumers_sync();  // the previous piece's values have been read
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float v = l[nt][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (nan) v = __int_as_float(0x7fc00000);
                if (gid == 0) {
                    sm[warp * kQ + nt * 8 + 2 * tig + e] = m[nt][e];
                    sl[warp * kQ + nt * 8 + 2 * tig + e] = v;
                }
            }
        consumers_sync();
        float M[NT][2], Lt[NT][2];  // of the piece, for query heads 2 tig, 2 tig + 1 of each n-tile
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int qi = nt * 8 + 2 * tig + e;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; w++) top = fmaxf(top, sm[w * kQ + qi]);
#pragma unroll
                for (int w = 0; w < kWarps; w++) sum += sl[w * kQ + qi] * weight_of(sm[w * kQ + qi], top);
                M[nt][e] = top, Lt[nt][e] = sum;
            }
        auto each = [&](auto f) {  // this lane's float4s in a warp's O, scaled
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const float f0 = weight_of(m[nt][0], M[nt][0]), f1 = weight_of(m[nt][1], M[nt][1]);
#pragma unroll
                for (int i = 0; i < D / 16; i++)
                    f((nt * (D / 16) + i) * 32 + lane, make_float4(o[nt][i][0] * f0, o[nt][i][1] * f1, o[nt][i][2] * f0,
                                                                  o[nt][i][3] * f1));
            }
        };
        float4 *buf = join + (warp & 1) * (kQ * D / 4);
        static_assert(kWarps == 4, "two rounds of two");
        if (warp >= 2) each([&](int at, float4 v) { buf[at] = v; });
        consumers_sync();
        if (warp < 2)
            each([&](int at, float4 v) {
                const float4 u = buf[at];
                buf[at] = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
            });
        consumers_sync();

        // ---- the piece's result: to the output, or to the workspace and, by the last, joined
        const float vs = kType ? __ldcg(p.v_scale + hk) : 1.f;
        constexpr int kPer = D / 64;  // float4s of a thread and n-tile
        auto store = [&](int nt, int j, float4 v, float2 lt) {
            // float4 (lane, block i): dimensions d and d + step of query heads qi, qi + 1
            const int i = j * kWarps + warp, qi = nt * 8 + 2 * tig;
            const int d = kType == 0 ? 16 * i + gid : 16 * i + 2 * gid, step = kType == 0 ? 8 : 1;
            uint16_t *at = p.out + (int64_t)b * p.ld_out + (head0 + qi) * D + d;
            // no keys: 0; keys whose scores are all -infinity have a sum of 0 too, and give 0 / 0
            const bool none = s.len == s.first && !s.bad;
            const float i0 = none ? 0.f : vs / lt.x, i1 = none ? 0.f : vs / lt.y;
            if (qi < nq) at[0] = float_to_half_bits(v.x * i0), at[step] = float_to_half_bits(v.z * i0);
            if (qi + 1 < nq) at[D] = float_to_half_bits(v.y * i1), at[D + step] = float_to_half_bits(v.w * i1);
        };
        auto store_lse = [&](int nt, float2 top, float2 lt) {
            if (!p.lse || warp != 0 || gid != 0) return;
            const int qi = nt * 8 + 2 * tig;
            float *at = p.lse + (int64_t)b * p.Hq + head0 + qi;
            if (qi < nq) at[0] = lt.x == 0.f ? -INFINITY : 0.69314718055994530942f * (top.x + (log2f(lt.x) - kLift));
            if (qi + 1 < nq) at[1] = lt.y == 0.f ? -INFINITY : 0.69314718055994530942f * (top.y + (log2f(lt.y) - kLift));
        };
        if (s.bad && warp == 0 && lane == 0) atomicOr(p.status, kDevStatusCacheRange);
        auto total_at = [&](int nt, int j) {
            const int at = (nt * (D / 16) + j * kWarps + warp) * 32 + lane;
            const float4 u = join[at], v = join[kQ * D / 4 + at];
            return make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
        };
        if (walk.t == 0 && end == s.tiles) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const float2 lt = make_float2(Lt[nt][0], Lt[nt][1]);
#pragma unroll
                for (int j = 0; j < kPer; j++) store(nt, j, total_at(nt, j), lt);
                store_lse(nt, make_float2(M[nt][0], M[nt][1]), lt);
            }
        } else {
            // slot 2c + 1: the piece that begins its item; slot 2c: one that continues it
            float *slot = p.partials + (2 * cta + (walk.t == 0 ? 1 : 0)) * kSlot;
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
#pragma unroll
                for (int j = 0; j < kPer; j++)
                    reinterpret_cast<float4 *>(slot)[(nt * (D / 16) + j * kWarps + warp) * 32 + lane] = total_at(nt, j);
                if (warp == 0 && gid == 0)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        slot[kQ * D + nt * 8 + 2 * tig + e] = M[nt][e];
                        slot[kQ * D + kQ + nt * 8 + 2 * tig + e] = Lt[nt][e];
                    }
            }
            // CTAs of the item's first and last unit: unit u lies in CTA ((u + 1) nc - 1) / W
            const int64_t u0 = w1 - walk.left - walk.t, u1 = u0 + s.tiles - 1;
            const int c_first = (int)divide((u0 + 1) * nc - 1, W), parts = (int)divide((u1 + 1) * nc - 1, W) - c_first + 1;
            auto slot_no = [&](int k) { return 2 * (c_first + k) + (k == 0 ? 1 : 0); };
            auto slot_at = [&](int k) { return p.partials + (int64_t)slot_no(k) * kSlot; };
            // counts this CTA's arrival; true for the last of `total`, which then sees all they wrote
            auto arrive = [&](unsigned int *counter, int total) -> bool {
                consumers_sync();
                if (tid == 0) {
                    unsigned int old;
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
                    last_flag = old == (unsigned int)(total - 1);
                    if (last_flag) *counter = 0u;  // for the next call
                }
                consumers_sync();
                return last_flag != 0;
            };
            // parts k0, k0 + step, .. below k1 of n-tile nt in one pass, kAhead of them read at a time:
            // running maximum and sums of the parts, as for the keys
            auto add_parts = [&](int k0, int k1, int step, int nt, float2 &top, float2 &lt, float4 (&acc)[kPer]) {
                constexpr int kAhead = 16 / kPer;
                const int qi = nt * 8 + 2 * tig;
                top = make_float2(-INFINITY, -INFINITY), lt = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kPer; j++) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = k0; k < k1; k += kAhead * step) {
                    float2 mm[kAhead], ll[kAhead];
                    float4 v[kAhead][kPer];
#pragma unroll
                    for (int u = 0; u < kAhead; u++) {  // (past the last: the first again, without weight)
                        const float *sp = slot_at(k + u * step < k1 ? k + u * step : k0);
                        mm[u] = load_now(reinterpret_cast<const float2 *>(sp + kQ * D + qi));
                        ll[u] = load_now(reinterpret_cast<const float2 *>(sp + kQ * D + kQ + qi));
#pragma unroll
                        for (int j = 0; j < kPer; j++)
                            v[u][j] = load_now(reinterpret_cast<const float4 *>(sp) +
                                               (nt * (D / 16) + j * kWarps + warp) * 32 + lane);
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; u++) {
                        if (k + u * step >= k1) mm[u] = make_float2(-INFINITY, -INFINITY), ll[u] = make_float2(0.f, 0.f);
                        const float2 t2 = make_float2(fmaxf(top.x, mm[u].x), fmaxf(top.y, mm[u].y));
                        const float g0 = weight_of(top.x, t2.x), g1 = weight_of(top.y, t2.y);
                        const float f0 = weight_of(mm[u].x, t2.x), f1 = weight_of(mm[u].y, t2.y);
                        top = t2;
                        lt.x = lt.x * g0 + ll[u].x * f0, lt.y = lt.y * g1 + ll[u].y * f1;
#pragma unroll
                        for (int j = 0; j < kPer; j++) {
                            acc[j].x = acc[j].x * g0 + v[u][j].x * f0, acc[j].y = acc[j].y * g1 + v[u][j].y * f1;
                            acc[j].z = acc[j].z * g0 + v[u][j].z * f0, acc[j].w = acc[j].w * g1 + v[u][j].w * f1;
                        }
                    }
                }
            };
            // Few parts: the last CTA of the item adds them all.  Many: in groups of about their
            // root, each added by its last CTA into the slot of its first part, then the groups
            // (one CTA reads 8 parts of 128 x 8 in about 1.1 us; a level costs about 1 us more).
            int group = parts;
            if (parts > kFlatParts) {
                group = (int)ceilf(sqrtf((float)parts));
                const int k0 = ((int)cta - c_first) / group * group, k1 = k0 + group < parts ? k0 + group : parts;
                if (arrive(p.counters + slot_no(k0), k1 - k0)) {
                    float2 top[NT], lt[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        float4 acc[kPer];
                        add_parts(k0, k1, 1, nt, top[nt], lt[nt], acc);
#pragma unroll
                        for (int j = 0; j < kPer; j++)
                            reinterpret_cast<float4 *>(slot_at(k0))[(nt * (D / 16) + j * kWarps + warp) * 32 + lane] = acc[j];
                    }
                    consumers_sync();  // every warp has read the first part's m and l
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
                        if (warp == 0 && gid == 0) {
                            float *sp = slot_at(k0) + kQ * D + nt * 8 + 2 * tig;
                            *reinterpret_cast<float2 *>(sp) = top[nt];
                            *reinterpret_cast<float2 *>(sp + kQ) = lt[nt];
                        }
                } else {
                    group = 0;  // nothing more to do here
                }
            }
            const int groups = group == 0 ? 0 : group == parts ? parts : (parts + group - 1) / group;
            if (groups > 0 && arrive(p.counters + 2 * gridDim.x + c_first, groups)) {
                const int step = group == parts ? 1 : group;
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float2 top, lt;
                    float4 acc[kPer];
                    add_parts(0, parts, step, nt, top, lt, acc);
#pragma unroll
                    for (int j = 0; j < kPer; j++) store(nt, j, acc[j], lt);
                    store_lse(nt, top, lt);
                }
            }
        }
        walk.next(p, end);
    }
}

constexpr int kMaxDevices = 64, kMaxCtasPerSm = 4;

// Sets an instance up on the current device and gives its resident CTAs per SM (both are properties
// of the instance and the device, looked up once; callers hold the library's lock).
template <int D, int kType, int NT>
cudaError_t prepare(int *per_sm) {
    static int known[kMaxDevices];
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (known[dev] == 0) {
        constexpr int smem = layout<D, kType, NT>().total;
        auto kern = attention_kernel<D, kType, NT>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        int n = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, smem);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        known[dev] = n < kMaxCtasPerSm ? n : kMaxCtasPerSm;
    }
    *per_sm = known[dev];
    return cudaSuccess;
}

// A pool as rows of kInner bytes: (byte, place in the page, 128-byte block, page and head).
cudaError_t encode_pool(CUtensorMap *map, const void *pool, const KvCache &c, int row_bytes, int inner, int tile) {
    EncodeTiledFn encode = encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const int slab = c.page_size < tile ? c.page_size : tile;
    const cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)c.page_size, (cuuint64_t)(row_bytes / inner),
                                (cuuint64_t)(c.pages * c.kv_heads)};
    const cuuint64_t strides[3] = {(cuuint64_t)row_bytes, (cuuint64_t)inner, (cuuint64_t)row_bytes * c.page_size};
    const cuuint32_t box[4] = {(cuuint32_t)inner, (cuuint32_t)slab, (cuuint32_t)(row_bytes / inner), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(pool), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int kType, int NT>
cudaError_t launch(Params &p, const KvCache &c, cudaStream_t s, const DeviceInfo &dev) {
    using C = Cfg<D, kType, NT>;
    CUtensorMap k_map, v_map;
    cudaError_t e = encode_pool(&k_map, c.k, c, C::kRowBytes, C::kInner, C::kTile);
    if (e == cudaSuccess) e = encode_pool(&v_map, c.v, c, C::kRowBytes, C::kInner, C::kTile);
    int per_sm = 0;
    if (e == cudaSuccess) e = prepare<D, kType, NT>(&per_sm);
    if (e != cudaSuccess) return e;
    p.GT = (p.G + 8 * NT - 1) / (8 * NT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(per_sm * dev.sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = layout<D, kType, NT>().total;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_kernel<D, kType, NT>, k_map, v_map, p);
}

}  // namespace

size_t attention_workspace_bytes(int64_t D, int64_t G, const DeviceInfo &dev) {
    const size_t slot = (size_t)(G > 8 ? 16 : 8) * (size_t)(D + 2) * sizeof(float);
    return (size_t)dev.sm_count * kMaxCtasPerSm * 2 * slot;
}

cudaError_t launch_paged_attention(const uint16_t *q, const KvCache &c, const int32_t *table, const int32_t *lengths,
                                   uint16_t *out, float *lse, int64_t B, int64_t Hq, int64_t ld_q, int64_t ld_out,
                                   int64_t width, int64_t window, float scale, const Workspace &ws, cudaStream_t s,
                                   const DeviceInfo &dev) {
    const int64_t G = Hq / c.kv_heads;
    if (ws.data_bytes < attention_workspace_bytes(c.head_dim, G, dev) || 3 * dev.sm_count * kMaxCtasPerSm > kMaxTiles)
        return cudaErrorInvalidValue;
    Params p = {};
    p.q = q;
    p.k_scale = c.k_scale, p.v_scale = c.v_scale;
    p.table = table, p.lengths = lengths;
    p.out = out, p.lse = lse;
    p.partials = reinterpret_cast<float *>(ws.data);
    p.counters = ws.counters;
    p.status = reinterpret_cast<unsigned int *>(ws.zeroed) + kCtlStatus;
    p.ld_q = ld_q, p.ld_out = ld_out, p.width = width, p.window = window;
    p.cap = width * c.page_size;
    p.B = (int)B, p.Hq = (int)Hq, p.Hkv = c.kv_heads, p.G = (int)G;
    p.pages = (int)c.pages;
    while ((1 << p.page_shift) < c.page_size) p.page_shift++;
    p.scale = scale;
    p.force_timeouts = dev.force_wait_timeouts;
    p.wait_limit = dev.force_wait_timeouts ? kForcedWaitPolls : kSpinLimit;
    auto by_queries = [&](auto one, auto two) { return G > 8 ? two(p, c, s, dev) : one(p, c, s, dev); };
    if (c.type == 0)
        return c.head_dim == 64    ? by_queries(launch<64, 0, 1>, launch<64, 0, 2>)
               : c.head_dim == 128 ? by_queries(launch<128, 0, 1>, launch<128, 0, 2>)
                                   : by_queries(launch<256, 0, 1>, launch<256, 0, 2>);
    return c.head_dim == 64    ? by_queries(launch<64, 1, 1>, launch<64, 1, 2>)
           : c.head_dim == 128 ? by_queries(launch<128, 1, 1>, launch<128, 1, 2>)
                               : by_queries(launch<256, 1, 1>, launch<256, 1, 2>);
}

}  // namespace bonsai

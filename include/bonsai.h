/*
 * bonsai.h -- C ABI of libbonsai, the B200 (sm_100a) ternary linear layer of
 * Bonsai 2-style ternary language models.
 *
 * The layer computes  y = x' . Wdeq^T  where
 *   - W is N x K (out x in) with trits t in {-1, 0, +1} and one FP16 scale per
 *     run of 128 weights along K:  Wdeq[n][k] = s[n][k/128] * t[n][k];
 *     source: "27B 模型压到 5.95GB，推理能力还保住 98%" (allhereai.com), the
 *     paragraph describing the method (ternary weights, a shared FP16 scale per
 *     128 weights, a block Hadamard rotation folded into storage);
 *   - x' = blockdiag(Hn) x is the online block-Hadamard rotation of the
 *     activations, Hn = H_128 / sqrt(128) with H_128 the Sylvester matrix
 *     (Hn[i][j] = (-1)^popcount(i & j) / sqrt(128)), applied to each run of 128
 *     activations starting at a multiple of 128; sources: the same page, the
 *     paragraph on running the files (a Hadamard activation runtime is needed,
 *     without it the output is garbage), and "Bonsai 2，把27B压进6个G"
 *     (10100.com), section 它怎么做到的 (the input must get the matching transform).
 *
 * Layouts (all row-major, all buffers owned by the caller):
 *   x       M x K   FP16 (IEEE binary16 bit patterns in uint16_t)
 *   y       M x N   FP16, round-to-nearest-even from an FP32 accumulator
 *   scales  N x K/128  FP16 (N x K/64 for BONSAI_FMT_PQ2_0_G64)
 *   trits   N x K   int8 in {-1, 0, +1}
 *   packed  the plane of one of the formats below: the two packings of the
 *           allhereai.com page (paragraph on the two file packings) and two
 *           variants the wmrh.cn page names:
 *     BONSAI_FMT_PTQ1_0  "compact trits", 1.75 bits/weight with the scale:
 *         row n, group g (128 weights) occupies 26 bytes at (n*K/128 + g)*26;
 *         byte b < 25 holds weights 128g+5b .. 128g+5b+4, byte 25 the last
 *         three, as  byte = sum_i (t_i + 1) * 3^i  (first weight least
 *         significant; padding digits zero, so byte 25 < 27; bytes >= 243
 *         are invalid).  Trit plane size N * K/128 * 26 bytes.
 *     BONSAI_FMT_PQ2_0   one trit per 2-bit slot, 2.125 bits/weight with the
 *         scale: weight k of row n is code t+1 in bits 2(k%4), 2(k%4)+1 of byte
 *         n*K/4 + k/4 (code 3 is invalid).  Trit plane size N * K/4 bytes.
 *     BONSAI_FMT_Q1_0    the 1-bit sibling of the wmrh.cn page (section 核心观点,
 *         ~1.125 bits/weight; section 关键机制, weights in {-1, +1} with an FP16
 *         group scale): weight k of row n is bit k%8 of byte n*K/8 + k/8, 1 for +1
 *         and 0 for -1 (every byte is valid).  Plane size N * K/8 bytes.  Same
 *         scale plane and the same rotation of x as the ternary packings.
 *     BONSAI_FMT_PQ2_0_G64  the PQ2_0 plane (same bytes, packed by bonsai_pack_pq2)
 *         with one FP16 scale per 64 weights: scales is N x K/64, scale g covering
 *         weights 64g .. 64g+63 of its row (the pages' Q2_0_g64; wmrh.cn page, 快速上手
 *         and 后端支持现状).  2.25 bits/weight with the scales.
 *
 * Conventions for every entry point:
 *   - Pointers are CUDA device pointers (any allocator) and must be 16-byte
 *     aligned, unless an entry point says otherwise; sizes are element counts.  K must be a
 *     positive multiple of 128; M and N must be >= 1 (M = 0 or N = 0 is accepted and
 *     launches nothing; so are T = 0 and B = 0).
 *   - stream is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Calls are asynchronous on it.  The return value reports argument
 *     validation and launch only: on a non-zero return nothing was launched
 *     (validation) or the launch failed (BONSAI_ERR_CUDA).  Faults inside a
 *     kernel surface at the caller's next synchronisation.
 *   - The library keeps one internal workspace per device (FP32 split-K
 *     partials, an FP16 copy of x' for the prefill GEMM, the partial results of
 *     bonsai_paged_attention).  It is allocated
 *     with cudaMalloc on the first call that needs it, grown when a larger
 *     call arrives (with a device synchronisation), and released by
 *     bonsai_shutdown().  Calls that use it must not overlap on the GPU (keep
 *     them on one stream); bonsai_reserve() sizes it ahead of stream capture.
 *     A workspace that a larger one replaces is kept until bonsai_shutdown(), so
 *     that captured calls stay valid; replay none after it.
 *   - Invalid codes in a packed plane (PTQ1_0 bytes >= 243, PQ2_0 code 3)
 *     produce unspecified output values but never out-of-bounds accesses.
 *   - Every wait inside a kernel (a barrier on a copy in flight, a hand-over
 *     between CTAs of the same grid) gives up after a bounded number of polls;
 *     the call then writes NaN to the outputs it could not finish instead of
 *     hanging the GPU, and sets a bit in the device status word that
 *     bonsai_device_status() reads.  Hand-over data carries the number of the call
 *     that wrote it, so a piece that arrives after its reader gave up is never taken
 *     for a later call's: the next call runs normally.
 */
#ifndef BONSAI_H
#define BONSAI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BONSAI_FMT_PTQ1_0 = 1,
    BONSAI_FMT_PQ2_0 = 2,
    BONSAI_FMT_Q1_0 = 3,
    BONSAI_FMT_PQ2_0_G64 = 4
} bonsai_fmt;

typedef enum {
    BONSAI_OK = 0,
    BONSAI_ERR_NULL = -1,   /* a required pointer is NULL                          */
    BONSAI_ERR_SHAPE = -2,  /* M, N or K negative, K not a multiple of 128, or too large */
    BONSAI_ERR_FMT = -3,    /* unknown packing format                             */
    BONSAI_ERR_ALIGN = -4,  /* a pointer is not 16-byte aligned                   */
    BONSAI_ERR_CUDA = -5,   /* a CUDA runtime call or kernel launch failed        */
    BONSAI_ERR_ARCH = -6,   /* the current device is not compute capability 10.0  */
    BONSAI_ERR_NOMEM = -7,  /* the internal workspace could not be allocated      */
    BONSAI_ERR_ALGO = -8,   /* the requested kernel cannot run this shape         */
    BONSAI_ERR_TOO_LARGE = -9, /* beyond the fixed scratch of bonsai_ternary_linear_noalloc */
    BONSAI_ERR_ARG = -10    /* an unknown activation, layout, scaling or cache type, or a
                               parameter outside its range                        */
} bonsai_status;

/* Kernel selection for bonsai_ternary_linear_algo (bonsai_ternary_linear uses AUTO). */
typedef enum {
    BONSAI_ALGO_AUTO = 0,
    BONSAI_ALGO_SIMPLE = 1,  /* one warp per output row; any M (slow, plain)              */
    BONSAI_ALGO_GEMV = 2,    /* batch-1 lookup-table GEMV with split-K; M == 1 only       */
    BONSAI_ALGO_SKINNY = 3,  /* register-dequant tensor-core kernel; 1 <= M <= 16         */
    BONSAI_ALGO_GEMM = 4,    /* tcgen05/TMEM prefill GEMM on FP16 tiles; any M            */
    BONSAI_ALGO_IMMA = 5     /* GEMV on the integer tensor cores, PQ2_0 and PQ2_0 g64:
                                M == 1 (K <= 24576), M == 2 (K <= 12288), and for
                                PQ2_0 M == 3 (K <= 6144)                                  */
} bonsai_algo;

/* Library version, (major << 16) | (minor << 8) | patch. */
int bonsai_version(void);

/* Human-readable text for a bonsai_status value (static storage). */
const char *bonsai_status_string(int status);

/* BONSAI_OK if the current CUDA device is an sm_100 part the library was compiled for,
 * BONSAI_ERR_ARCH if it is another architecture, BONSAI_ERR_CUDA if there is no
 * usable device. */
int bonsai_check_device(void);

/* Bytes of the packed trit plane for N x K weights (scales excluded: they are
 * N * K/128 FP16 values, N * K/64 for BONSAI_FMT_PQ2_0_G64).  Returns BONSAI_ERR_SHAPE / BONSAI_ERR_FMT
 * (negative) on a bad argument. */
int64_t bonsai_packed_bytes(int fmt, int64_t N, int64_t K);

/* Packs N x K trits into the PTQ1_0 plane (layout above).  A trit outside
 * {-1, 0, +1} makes its byte 0xFF, an invalid code, so a bad input is
 * detectable by bonsai_unpack.  Packing is an offline step; its cost is not on
 * the inference path.  Source: allhereai.com page, paragraph on the packings. */
int bonsai_pack_ptq1(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream);

/* Packs N x K trits into the PQ2_0 plane (layout above).  A trit outside
 * {-1, 0, +1} is stored as the invalid code 3.  Same source. */
int bonsai_pack_pq2(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream);

/* Packs N x K weights into the Q1_0 plane (layout above): +1 -> bit 1, any other
 * value -> bit 0 (-1).  Source: wmrh.cn page, sections 核心观点 and 关键机制. */
int bonsai_pack_q1(const int8_t *trits, uint8_t *packed, int64_t N, int64_t K, void *stream);

/* Unpacks a plane of format fmt back into N x K int8 trits.  Invalid codes
 * unpack to -128 (every trit of an invalid PTQ1_0 byte).  Test hook: it makes
 * the packed layout checkable byte for byte. */
int bonsai_unpack(int fmt, const uint8_t *packed, int8_t *trits, int64_t N, int64_t K,
                  void *stream);

/* x_out = blockdiag(Hn) x for an M x K FP16 matrix (the rotation defined above),
 * computed in FP32 and rounded to FP16 (nearest even).  x_out may equal x (in
 * place) but must not otherwise overlap it.  This is the same transform
 * bonsai_ternary_linear applies internally; it is exported for callers that
 * keep rotated activations and as a test hook. */
int bonsai_hadamard128(const uint16_t *x, uint16_t *x_out, int64_t M, int64_t K, void *stream);

/* y = x' . Wdeq^T (definitions above) for un-rotated FP16 x: the Hadamard
 * rotation of x is applied inside the call.  Dispatch on M: M == 1 -> the
 * integer tensor-core GEMV (PQ2_0 and PQ2_0 g64, K <= 24576, and a grid of at most one
 * CTA per SM: up to about 14,000 items of 32 rows x 512 weights on 148 SMs) or the lookup-table GEMV
 * (PTQ1_0, Q1_0), 2 <= M <= 16 -> skinny tensor-core kernel (PQ2_0, PQ2_0 g64,
 * Q1_0), otherwise (and for PTQ1_0 at 2 <= M <= 16) the tcgen05 GEMM.  The
 * integer GEMV holds each 128-group of x' as 16-bit fixed point with a power-of-two
 * scale (|x~| <= 2^14) before the exact integer products; the other kernels round
 * x' to FP16 (GEMM, skinny) or keep it in FP32 (lookup tables, plain kernel).  y must
 * not overlap x, packed or scales.  Source of the operation: allhereai.com page,
 * method paragraph and packings paragraph. */
int bonsai_ternary_linear(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                          uint16_t *y, int64_t M, int64_t N, int64_t K, int fmt, void *stream);

/* As bonsai_ternary_linear with an explicit kernel choice (bonsai_algo) and an
 * explicit split-K factor for the skinny kernel (0 = automatic, 1 = no split,
 * otherwise the number of K chunks, clamped to what the shape allows).  For
 * BONSAI_ALGO_GEMM the same argument picks the M tile instead: 1 = 128 rows per CTA,
 * 2 = 256 rows (two TMEM accumulators sharing each expanded weight tile), 3 = CTA
 * pairs (clusters of two SMs issuing 256-row tcgen05 MMAs together, each SM expanding
 * half of every weight tile; an explicit choice only), 0 = automatic (1 or 2).  For
 * BONSAI_ALGO_GEMV it picks the schedule: 1 = each CTA walks all K slices of its rows
 * (no split-K), >= 2 = one 512-wide K slice per CTA with split-K partials, 0 =
 * automatic.  BONSAI_ALGO_IMMA ignores it (its work split is fixed
 * by the shape and the SM count, so results are bitwise repeatable).
 * Returns BONSAI_ERR_ALGO if the chosen kernel cannot run the shape (e.g.
 * BONSAI_ALGO_GEMV with M > 1, or BONSAI_ALGO_IMMA on a shape whose grid would not fit
 * on the current device at once, the limit the automatic choice also applies).  For
 * measurement and testing of each kernel. */
int bonsai_ternary_linear_algo(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                               uint16_t *y, int64_t M, int64_t N, int64_t K, int fmt, int algo,
                               int split_k, void *stream);

/* The SwiGLU step of the MLP after a fused gate/up projection: for y, the M x 2F FP16
 * output of a linear layer whose weight rows 0 .. F-1 are the gate projection and
 * F .. 2F-1 the up projection, h[m][f] = silu(y[m][f]) * y[m][F + f] with
 * silu(z) = z / (1 + e^-z), computed in FP32 and rounded to FP16 (nearest even).  h is
 * M x F; y and h must not overlap.  Source of the fused gate/up projection: the
 * 27B-class layer shapes (d = 5120, ffn = 17408, gate/up N = 34816). */
int bonsai_swiglu(const uint16_t *y, uint16_t *h, int64_t M, int64_t F, void *stream);

/* The fused gate/up linear layer followed by SwiGLU: packed and scales hold 2F weight rows
 * (gate rows first, then up rows: the N = 2F plane of bonsai_ternary_linear) and h gets
 * the M x F result of bonsai_swiglu applied to their product with x'.  On the integer
 * tensor-core GEMV (PQ2_0 and PQ2_0 g64 at the batches and K it takes: see
 * BONSAI_ALGO_IMMA) and the prefill GEMM the step runs in the kernel's epilogue on the
 * FP32 sums; the lookup-table GEMV, the skinny and the plain kernel write the product to
 * the library's workspace in FP16 and bonsai_swiglu follows. */
int bonsai_ternary_linear_swiglu(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                                 uint16_t *h, int64_t M, int64_t F, int64_t K, int fmt, void *stream);

/* Activations of bonsai_ternary_linear_epilogue. */
typedef enum {
    BONSAI_ACT_NONE = 0,
    BONSAI_ACT_RELU = 1,     /* max(z, 0)                                             */
    BONSAI_ACT_SILU = 2,     /* z / (1 + e^-z)                                        */
    BONSAI_ACT_GELU = 3,     /* z (1 + erf(z / sqrt 2)) / 2                           */
    BONSAI_ACT_GELU_TANH = 4 /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2       */
} bonsai_act;

/* y = act(x' . Wdeq^T + bias) + residual in one call: the product of bonsai_ternary_linear
 * with its bias, activation and residual stream applied to the FP32 sums, rounded to FP16
 * once.  bias: N FP16 values, or NULL for none; residual: M x N FP16, or NULL for none; act:
 * a bonsai_act.  residual may be y itself (the residual stream updated in place) but must
 * not overlap y otherwise; y must not overlap x, packed, scales or bias.  algo and split_k
 * choose the kernel as in bonsai_ternary_linear_algo, except that the skinny kernel takes
 * batches of up to 1024 tokens here (in groups of 16), which the automatic choice
 * (BONSAI_ALGO_AUTO and 0) uses for small layers, and that the GEMM's CTA pairs
 * (split_k = 3) are not available and return BONSAI_ERR_ALGO, whoever chose the GEMM.  An
 * unknown act returns BONSAI_ERR_ARG.  The activations are computed in FP32; GELU's erfc is off by
 * up to 1.5e-7, which near z = -4 comes to 1.25 half steps of FP16 ahead of the rounding.  A NaN
 * sum (that of a wait that gave up, for instance) stays a NaN through every activation.  The pages describe no such step: the projections of a decoder
 * layer add biases and the residual stream here. */
int bonsai_ternary_linear_epilogue(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                                   const uint16_t *bias, const uint16_t *residual, uint16_t *y, int64_t M,
                                   int64_t N, int64_t K, int fmt, int act, int algo, int split_k, void *stream);

/* Which elements of a head form the pairs that a rotary position turns: the first R of the
 * head's D elements are rotated, the rest pass unchanged. */
typedef enum {
    BONSAI_ROPE_HALF = 0,       /* (i, i + R/2) for i < R/2 */
    BONSAI_ROPE_INTERLEAVED = 1 /* (2i, 2i + 1) for i < R/2 */
} bonsai_rope_layout;

/* How the frequencies of the pairs are stretched for contexts longer than the trained one
 * (bonsai_rope_frequencies); f_i = base^(-2i/R). */
typedef enum {
    BONSAI_ROPE_PLAIN = 0,  /* f_i                                                        */
    BONSAI_ROPE_LINEAR = 1, /* f_i / factor                                               */
    BONSAI_ROPE_NTK = 2,    /* f_i with the base times factor^(R / (R - 2))               */
    BONSAI_ROPE_YARN = 3,   /* f_i / factor for pairs turning fewer than `low` times over
                               `original` positions, f_i for those turning more than
                               `high` times, a linear ramp over the pair index between;
                               magnitude 1 + 0.1 ln(factor)                               */
    BONSAI_ROPE_BANDS = 4   /* the same two ends, and between them f_i (1 - s) / factor +
                               f_i s with s linear in the number of turns                 */
} bonsai_rope_scaling;

/* The frequencies of rotary positions, computed on the HOST in FP64: freqs[i], i < R/2, in
 * radians per position, and the factor *magnitude on the rotated values (1 but for YARN).
 * freqs and magnitude are HOST pointers; the caller copies freqs to the device for
 * bonsai_rope and bonsai_rope_append.  R even and >= 0, base > 1, factor >= 1 (scalings 1 to
 * 4), original > 0 and 0 < low < high (YARN and BANDS; otherwise ignored); all finite, or
 * BONSAI_ERR_ARG.  R odd or negative returns BONSAI_ERR_SHAPE.  Needs no GPU. */
int bonsai_rope_frequencies(double *freqs, double *magnitude, int64_t R, double base, int scaling,
                            double factor, double original, double low, double high);

/* Rotary positions: turns each pair (a, b) of each head's first R elements by the angle
 * positions[t] * freqs[i],
 *   (a, b) -> magnitude * (a cos - b sin, b cos + a sin),
 * the angle in FP64 (reduced to one turn there, so that far positions lose nothing), the
 * sine and cosine and the products in FP32, one rounding to FP16.  x and out hold T rows of
 * H heads of D FP16 elements; row t starts at element t * ld_x (t * ld_out), so that the
 * query and key heads of a fused projection's output are rotated where they lie.  out may
 * be x with ld_out = ld_x (in place; one row has no stride) but must not overlap it otherwise;
 * elements between H * D and the row stride are not touched.  freqs: R/2 FP64 values, positions: T int32
 * values, both device memory aligned to their element.  D a positive multiple of 8 up to
 * 1024; R even, 0 <= R <= D (R = 0 copies; freqs may then be NULL); ld_x and ld_out at least
 * H * D and multiples of 8.  No workspace. */
int bonsai_rope(const uint16_t *x, uint16_t *out, const double *freqs, const int32_t *positions,
                int64_t T, int64_t H, int64_t D, int64_t R, int64_t ld_x, int64_t ld_out,
                float magnitude, int layout, void *stream);

/* Element types of a paged key/value cache. */
typedef enum {
    BONSAI_KV_F16 = 0, /* FP16                                                             */
    BONSAI_KV_E4M3 = 1 /* 8-bit floats (4 exponent, 3 mantissa bits) times a positive FP32
                          scale per key/value head: k_scale and v_scale, Hkv values each    */
} bonsai_kv_type;

/* A paged key/value cache is two pools, k_cache and v_cache, of `pages` pages each:
 *   pages x Hkv x page_size x D elements of kv_type, row-major,
 * so that one head's keys of one page are page_size * D contiguous elements.  Position j of
 * a sequence lies in entry j / page_size of its row of the page table, at place
 * j % page_size of that page.  page_size is 16, 32, 64, 128 or 256; D 64, 128 or 256;
 * pages < 2^31.  k_scale and v_scale are read for BONSAI_KV_E4M3 only (NULL otherwise).
 *
 * bonsai_rope_append turns one qkv projection's output into the new tokens' queries and
 * cache entries: row t of qkv (at element t * ld_qkv) holds Hq query heads, Hkv key heads
 * and Hkv value heads of D elements.  The query heads are rotated as by bonsai_rope into
 * row t of q_out (at t * ld_q); the key heads are rotated and the value heads copied to
 * slot slots[t] = page * page_size + place of the pools.  FP16 entries are rounded once
 * from FP32; E4M3 entries are value / scale, rounded to nearest even and saturated at
 * +-448 (a NaN stays one).  A negative slot writes no cache entry (a padded row); a slot of
 * pages * page_size or more writes none either and sets BONSAI_DEVICE_CACHE_RANGE in the
 * device status word.  Two tokens of one call must not share a slot.  q_out may be qkv with
 * ld_q = ld_qkv (the query heads then rotated in place; one row has no stride) but must not
 * overlap it otherwise.
 * Hq >= 0, a multiple of Hkv; ld_qkv >= (Hq + 2 Hkv) * D and ld_q >= Hq * D, multiples of
 * 8; positions (int32), slots (int64), freqs (FP64) and the scales aligned to their
 * element.  freqs, R, magnitude and layout as for bonsai_rope.  Uses the control words of
 * the workspace only (the status bit), so it may overlap other calls. */
int bonsai_rope_append(const uint16_t *qkv, uint16_t *q_out, void *k_cache, void *v_cache,
                       const float *k_scale, const float *v_scale, const double *freqs,
                       const int32_t *positions, const int64_t *slots, int64_t T, int64_t Hq, int64_t Hkv,
                       int64_t D, int64_t R, int64_t ld_qkv, int64_t ld_q, int64_t pages, int64_t page_size,
                       float magnitude, int layout, int kv_type, void *stream);

/* Attention of one new token per sequence over a paged cache:
 *   out[b][h] = sum_j p_j v_j,  p = softmax_j(scale * q[b][h] . k_j),
 * over the positions j of sequence b with max(0, lengths[b] - window) <= j < lengths[b]
 * (window = 0: all of them; the new token's own entry is appended before the call and
 * counted in lengths).  Query head h reads key/value head h / (Hq / Hkv).  q and out hold B
 * rows of Hq heads of D FP16 elements at row strides ld_q and ld_out; out must not overlap
 * q or the cache.  lse (may be NULL) gets the B x Hq FP32 natural logarithms of the sums of
 * e^(scale q.k), so that results over parts of a context can be joined.  A sequence of
 * length 0 gives zeros and an lse of -infinity; one whose scores are all -infinity gives
 * NaN, as the formula does.
 *   page_table: B rows of max_pages int32 page numbers; entries past a sequence's last page
 * (and before its window) are not read.  lengths: B int32 values.  Entries of the cache at
 * other positions (the rest of the last page, freed pages) are never part of a result,
 * whatever bits they hold.  A page number outside [0, pages) for a page in use, or a length
 * that is negative or exceeds max_pages * page_size, makes that sequence's outputs NaN and
 * sets BONSAI_DEVICE_CACHE_RANGE; nothing outside the buffers is read.
 *   Statistics, scores and sums are FP32; the probabilities are rounded to FP16 before the
 * product with the values (2^-11 of each; below 2^-28 of a sequence's largest, 2^-39 of that).
 * Results depend on the lengths and the device's SM count only (bitwise repeatable).  Hq a positive multiple of Hkv; ld_q, ld_out at least Hq * D and
 * multiples of 8; page_table, lengths, lse and the scales aligned to their element; window
 * >= 0.  Uses the workspace: see the conventions above (less of it than bonsai_reserve makes
 * for any shape). */
int bonsai_paged_attention(const uint16_t *q, const void *k_cache, const void *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *page_table, const int32_t *lengths,
                           uint16_t *out, float *lse, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                           int64_t ld_q, int64_t ld_out, int64_t pages, int64_t page_size, int64_t max_pages,
                           int64_t window, float scale, int kv_type, void *stream);

/* Number of kernels one bonsai_ternary_linear_algo call with these arguments launches
 * on the current device (the lookup-table GEMV: 1, or 2 when its split-K partials are
 * summed by a second kernel; the integer tensor-core GEMV: 1; the other kernels: 2,
 * the rotation pass and the kernel),
 * or a negative bonsai_status.  Launches nothing. */
int bonsai_launch_count(int64_t M, int64_t N, int64_t K, int fmt, int algo, int split_k);

/* Grows the calling device's workspace so that calls up to M x N x K (any
 * format and kernel) need no further allocation; call before capturing calls
 * into a CUDA graph.  Synchronises the device if it reallocates. */
int bonsai_reserve(int64_t M, int64_t N, int64_t K);

/* Batch-1 ternary linear layer that allocates nothing.
 *
 * Some callers cannot call cudaMalloc: code that runs while a CUDA graph is being
 * captured, allocators that must own every byte on the device, or hosts that forbid
 * allocation after start-up.  This entry point computes the same y as
 * bonsai_ternary_linear for M == 1 with the split-K lookup-table GEMV, but takes that
 * kernel's scratch -- one FP32 partial sum per (512-weight K slice, output row) -- from
 * one fixed array in device memory that is part of the library image, instead of the
 * per-device workspace.  It never calls cudaMalloc, cudaFree or any allocating routine.
 * The pages this library follows describe no such variant: it exists only for these
 * callers.
 *
 * Formats: BONSAI_FMT_PTQ1_0 and BONSAI_FMT_PQ2_0 only; BONSAI_FMT_Q1_0 and
 * BONSAI_FMT_PQ2_0_G64 return BONSAI_ERR_FMT.
 * Limits: M must be 1, K a multiple of 512 and (K / 512) * N <= 1048576 (the array holds
 * 2^20 FP32 partials, 4 MiB, kept by every GPU that loads the library until the process
 * exits); other shapes return BONSAI_ERR_TOO_LARGE and launch nothing.  Checks run in
 * the order format, shape, NULL pointer, alignment, then these limits.  Inputs and
 * output are caller-owned device memory as for bonsai_ternary_linear.
 *
 * Set-up: the first call on each device looks up that device's copy of the array
 * (with that device current); make that first call before capturing any stream.
 * Every call shares the one array and leaves its partial sums there; each call writes
 * every partial it reads before reading it, so nothing needs clearing between calls.
 * Calls whose work overlaps on the GPU (different streams, or concurrent host threads)
 * race on the array -- serialise them. */
int bonsai_ternary_linear_noalloc(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                                  uint16_t *y, int64_t M, int64_t N, int64_t K, int fmt, void *stream);

/* Device status bits, set by a kernel whose bounded wait gave up (the call then wrote
 * NaN for the outputs it could not finish; see the conventions above), or that met a slot,
 * page or length outside the cache.  They stay set until cleared by bonsai_device_status. */
#define BONSAI_DEVICE_GEMV_COPY_TIMEOUT 1u  /* integer GEMV: a weight copy never landed      */
#define BONSAI_DEVICE_GEMV_PIECE_TIMEOUT 2u /* integer GEMV: a split tile's later piece, or  */
                                            /* its hand-over, never came                      */
#define BONSAI_DEVICE_GEMM_TIMEOUT 4u       /* prefill GEMM: a barrier or hand-over wait gave up */
#define BONSAI_DEVICE_SKINNY_TIMEOUT 8u     /* skinny kernel: the wait after the rotation   */
                                            /* phase, or a weight copy, never ended           */
#define BONSAI_DEVICE_CACHE_RANGE 16u       /* append or attention: a slot, page or length  */
                                            /* outside the cache (no such entry was touched)  */
#define BONSAI_DEVICE_ATTENTION_TIMEOUT 32u /* attention: a copy of keys and values never    */
                                            /* landed                                         */

/* Reads the calling device's status bits into *bits after synchronising `stream` (the
 * stream of the calls in question), and clears them when `clear` is non-zero.  *bits is 0
 * when no call has run on the device yet.  Returns BONSAI_ERR_NULL for a NULL bits,
 * BONSAI_ERR_CUDA if the copy or the synchronisation fails.  The pages describe no such
 * call; it reports the bounded waits of this implementation. */
int bonsai_device_status(void *stream, uint32_t *bits, int clear);

/* Test hook.  While enabled (enable != 0), the waits of the integer tensor-core GEMV for
 * the later pieces of its split row tiles, and of the prefill GEMM for its hand-over
 * flags, look for a call number that no CTA writes and give up after 64 polls; so does the
 * skinny kernel's wait after its rotation phase, whatever has arrived, and those of
 * bonsai_paged_attention wait as long for a copy that nobody makes.  The calls
 * then write NaN for those tiles (the last two: everywhere but for sequences without keys) and
 * set the status bits, without any fault, so that the timeout path can be tested.  Off by default;
 * applies to calls launched while enabled. */
int bonsai_debug_force_timeouts(int enable);

/* Frees the workspaces of every device (after synchronising each).  The
 * library stays usable: the next call allocates again. */
void bonsai_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* BONSAI_H */

/*
 * lowbit.h -- C ABI of liblowbit.so: products of packed low-bit weights with int8 activations on one
 * AMD Instinct MI355X (gfx950).
 *
 * Weight formats:
 *   LB_Q1_0           ggml Q1_0: 18-byte blocks of 128 weights, binary16 scale d then 16 bytes of sign
 *                     bits, least-significant bit first; weight = d * (bit ? +1 : -1).
 *                     (bankml technical report, section III.2 "The Q1_0 format and its arithmetic".)
 *   LB_Q2_0_G64       ggml Q2_0 with group 64: 18-byte blocks of 64 weights, binary16 d then 16 bytes of
 *                     2-bit codes, lowest bits first; weight = (code - 1) * d, code in {0,1,2,3}.
 *                     (bankml technical report, section III.5 "The Q2_0_g64 (ternary) kernel".)
 *   LB_TERNARY_PLANAR the planar ternary beat: 16 bytes per 64 consecutive columns of one row,
 *                     {u64 pos, u64 neg}, column c at bit c; weight = pos_c - neg_c, times one fp32
 *                     per-tensor scale.  (tritium "Architecture", section 2 "bit planes".)
 *   LB_Q8_0           ggml Q8_0 weights: 34-byte blocks of 32 weights, binary16 scale d then 32 signed
 *                     bytes; weight = d * byte.  The q8_0 block of the bankml technical report, section
 *                     III.2, used for weights ("Q8_0 weights" and vec_dot_q8_0_q8_0 for the KV cache in
 *                     the bankml build history's 0.3.9 entry).  Decode takes K up to 16384; prefill
 *                     (lowbit_gemm, lowbit_block_sums with M > 1) also needs K % 128 == 0 (LB_ESHAPE).
 *   LB_Q4_0           ggml Q4_0: 18-byte blocks of 32 weights, binary16 scale d then 16 bytes of 4-bit codes, byte j
 *                     holding weight j in its low and weight j + 16 in its high nibble; weight = (code - 8) * d.
 *                     Decode takes K up to 16384; prefill (lowbit_gemm, lowbit_block_sums with M > 1) also needs
 *                     K % 128 == 0 (LB_ESHAPE).
 *   LB_TERNARY_B3     base-3 ternary beats: 16 bytes per 80 consecutive columns of one row, byte j holding
 *                     columns 5j..5j+4 as the integer sum_t (w + 1) * 3^t, lowest digit first (0..242);
 *                     a row of K columns (K % 64 == 0) takes ceil(K/80) beats, the columns past K coded 0.
 *                     Weight = w times one fp32 per-tensor scale, with per-token int8 activations and the
 *                     planar output rule.  Five trits per byte (bankml technical report, section III.8
 *                     "Information"); base-3 packing of the planar body at 1.6 bits per weight (tritium
 *                     "Architecture", section 10).  Decode only; bytes above 242 are not base-3 bytes.
 *
 * Activation formats:
 *   LB_ACT_Q8_0       ggml q8_0: int8 xq[M][K] plus binary16 scales xscale[M][K/32]; one block of 32
 *                     activations per scale (bankml technical report, section III.2).  Used with the
 *                     ggml weight formats.
 *   LB_ACT_I8_ROW     int8 xq[M][K] plus one fp32 scale per row (per token), xscale[M] (tritium
 *                     "Architecture", section 1: activations are int8).  Used with the planar format.
 *   LB_ACT_F32_Q8_0   fp32 x[K], quantised to q8_0 by the batch itself, with exactly the arithmetic of
 *                     lowbit_quantize_act(LB_ACT_Q8_0) (so the results are bit-identical to quantising
 *                     first).  Batched decode of LB_Q1_0, LB_Q2_0_G64 and LB_Q4_0 only: a product that depends on the
 *                     previous one's output then needs no quantise call of its own.  Rows of at most 8192
 *                     columns are quantised inside the products' own launch (every workgroup quantises
 *                     the row it stages); a batch from lowbit_batch_create quantises longer rows with one
 *                     launch per distinct (x, K) ahead of its products, into device memory it owns.
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers unless stated otherwise; the caller owns every buffer.  No
 *     entry point below allocates, frees or synchronises, except lowbit_batch_create/destroy, which
 *     are set-up calls.
 *   - Work is enqueued asynchronously on the caller's HIP stream `s` (NULL = the null stream).
 *   - Arguments are validated on the host before anything is launched; an error launches nothing.
 *     There is no fallback path: an unsupported device or shape is an error, never a slower kernel.
 *   - Outputs are row-major fp32.  Integer per-block sums are exact; fp32 outputs follow the
 *     definition  y = sum_b d_w[b] * sum_{j in b} d_x[j] * isum[j]  up to fp32 rounding order.
 *   - N == 0 or M == 0 is an empty product: LB_OK, nothing launched.  K == 0 writes zeros.
 */
#ifndef LOWBIT_H
#define LOWBIT_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { LB_Q1_0 = 1, LB_Q2_0_G64 = 2, LB_TERNARY_PLANAR = 3, LB_Q8_0 = 4, LB_TERNARY_B3 = 5, LB_Q4_0 = 6 } lb_wfmt;
typedef enum { LB_ACT_Q8_0 = 1, LB_ACT_I8_ROW = 2, LB_ACT_F32_Q8_0 = 3 } lb_afmt;

typedef enum {
    LB_OK = 0,
    LB_EINVAL = 1,       /* null pointer, unknown enum, or a weight/activation format pairing that is not defined */
    LB_ESHAPE = 2,       /* negative size, K not a multiple of the weight block (128, 64, 64, 32, 64, 32), or over a limit */
    LB_EALIGN = 3,       /* a pointer is not aligned as its argument requires */
    LB_EUNSUPPORTED = 4, /* the current device is not gfx950, or the entry point has no kernel for the format */
    LB_EDEVICE = 5,      /* a HIP call failed; lowbit_last_error() holds the runtime's message */
    LB_ENOMEM = 6        /* host memory for a set-up object (lowbit_batch_create) could not be allocated */
} lb_status;

/* Human-readable name of a status code (static string). */
const char *lowbit_status_str(lb_status st);

/* Message of the last error raised by this library on the calling thread ("" if none; at most 511
 * characters, valid until the thread's next failing call). */
const char *lowbit_last_error(void);

/*
 * Bytes of the device layout of an N x K weight tensor in format `fmt`: 18 per Q1_0 / Q2_0_g64 / Q4_0 block (128,
 * 64 or 32 weights), 34 per Q8_0 block (32 weights), 16 per planar beat (64 columns) or base-3 beat (80
 * columns, ceil(K/80) per row) -- the same count as the on-disk format (1.125, 2.25, 4.5, 8.5, 2 and 1.6 bits
 * per weight; bankml technical report sections III.2, III.5 and III.8).
 * Returns -1 for a bad format or shape.
 */
int64_t lowbit_weight_bytes(int fmt, int64_t N, int64_t K);

/*
 * One-time conversion of a ggml block stream into the device layout the kernels read.
 *   blocks: device, N rows x K/QK blocks of 18 bytes (34 for Q8_0), row-major, no alignment requirement.
 *   packed: device, lowbit_weight_bytes(fmt, N, K) bytes, 16-byte aligned.  Layout: all 16-byte code
 *           records row-major ([N][K/QK][16]; Q8_0: 32-byte records of the block's weight bytes,
 *           [N][K/32][32]), then all binary16 scales row-major ([N][K/QK]).
 *           A Q2_0_g64 record is the block's 16 code bytes as they are.  A Q1_0 record permutes the
 *           block's 128 sign bits: the sign of weight 32r + 8m + k (r, m in 0..3, k in 0..7), at bit
 *           8m + k of little-endian dword r in the ggml block, sits at bit 4k + r of dword m, so one
 *           mask (0x11111111 << r) isolates eight weights of activation block r as nibbles.  A Q4_0 record holds
 *           weight 8k + n (k in 0..3, n in 0..7), in 4-bit two's complement, at bits 4n..4n+3 of dword k.
 * Lossless (lowbit_unpack_weights is its inverse).  For LB_TERNARY_PLANAR the beat stream already is
 * the device layout (tritium "Architecture", section 2: the file layout is the beat stream) and pack
 * copies it unchanged.  For LB_TERNARY_B3 pack keeps the beat stream and writes each base-3 byte v as
 * b = ceil(256 v / 243), whose leading m base-3 digits are floor(3^m b / 256) (unpack: v = 243 b >> 8).
 */
lb_status lowbit_pack_weights(int fmt, const void *blocks, int64_t N, int64_t K, void *packed, hipStream_t s);
lb_status lowbit_unpack_weights(int fmt, const void *packed, int64_t N, int64_t K, void *blocks, hipStream_t s);

/*
 * Quantise fp32 activation rows x[M][K] (device, 16-byte aligned).
 *   LB_ACT_Q8_0:  per block of 32, amax = max|x|; xscale (uint16 binary16, [M][K/32]) = fp16_rne(amax/127);
 *                 xq = round_half_even(x * (127/amax)) in fp32, 0 when amax = 0.  K % 32 == 0.
 *                 (bankml technical report, section III.2: 127 / max|x| with round-half-to-even.)
 *   LB_ACT_I8_ROW: per row, amax over the row; xscale (fp32, [M]) = amax/127;
 *                 xq = clamp(round_half_even(x * (127/amax)), -128, 127).
 *   xq: device int8 [M][K], 16-byte aligned.  xscale: device, 4-byte aligned.
 */
lb_status lowbit_quantize_act(int afmt, const float *x, int64_t M, int64_t K, int8_t *xq, void *xscale,
                              hipStream_t s);

/*
 * Batch-1 decode product y[N] = W . dequant(xq): the select-accumulate of the weights over the int8
 * activations, exact integer sums per activation block, scaled per block in fp32
 * (bankml technical report, sections III.2, III.5 and III.8; tritium "Architecture", sections 1-2).
 *   W:      device layout of the N x K tensor (lowbit_pack_weights; planar beats as they are), 16-byte aligned.
 *   w_tensor_scale: planar and base-3 per-tensor scale s_w (y = ((float)acc * s_x) * s_w); ignored otherwise.
 *   afmt:   LB_ACT_Q8_0 for the ggml formats, LB_ACT_I8_ROW for planar and base-3 beats.
 *   xq:     device int8 [K], 16-byte aligned.  xscale: binary16 [K/32] or one fp32, 4-byte aligned.
 *   y:      device fp32 [N], 4-byte aligned.
 * Limits: K <= 32768 (16384 for LB_Q4_0 and LB_Q8_0, 30720 for LB_TERNARY_B3) and N <= 2^31 - 1; the weight tensor must
 * be smaller than 4 GiB.
 */
lb_status lowbit_matvec(int fmt, const void *W, int64_t N, int64_t K, float w_tensor_scale, int afmt,
                        const int8_t *xq, const void *xscale, float *y, hipStream_t s);

/*
 * Prefill product Y[M][N] = dequant(Xq) . W^T for M activation rows: the same per-block integer sums
 * as lowbit_matvec, computed as int8 matrix-core products over weight tiles unpacked to int8 in LDS,
 * then scaled per block in fp32 (bankml technical report, section III.3: a tile that loads each weight
 * block once and applies it to several activation columns; tritium "Architecture", section 3:
 * prefill runs compute-bound).
 *   Xq: device int8 [M][K], 16-byte aligned; Xscale: binary16 [M][K/32] (ggml formats) or fp32 [M].
 *   Y:  device fp32 [M][N], 4-byte aligned.
 * Limits (else LB_ESHAPE): those of lowbit_matvec, M * N < 2^31 outputs, M * K < 2^32 activation bytes,
 * and K % 128 == 0 for LB_Q4_0 and LB_Q8_0.  LB_TERNARY_B3 has no prefill kernel (LB_EUNSUPPORTED).
 */
lb_status lowbit_gemm(int fmt, const void *W, int64_t N, int64_t K, float w_tensor_scale, int afmt,
                      const int8_t *Xq, const void *Xscale, int64_t M, float *Y, hipStream_t s);

/*
 * The exact integer sums the products above are built from, written by the same kernels (M == 1: the
 * decode kernel; M > 1: the prefill kernel) instantiated with one extra store:
 *   ggml formats: sums int32 [M][N][K/32], sums[m][n][j] = sum over activation block j of w * q;
 *   planar:       sums int32 [M][N], the whole row's select-accumulate.
 */
lb_status lowbit_block_sums(int fmt, const void *W, int64_t N, int64_t K, int afmt, const int8_t *Xq,
                            const void *Xscale, int64_t M, int32_t *sums, hipStream_t s);

/*
 * Dense bf16 head matvec y[N] = sum_k bf16_to_f32(W[n][k]) * x[k], accumulated in fp32
 * (tritium "Architecture", section 3: the dense head is the largest single stream; bf16 storage).
 *   W: device uint16 bf16 bits [N][K], 16-byte aligned, K % 8 == 0; x: device fp32 [K], 16-byte aligned;
 *   y: device fp32 [N].  K must be a multiple of 8 and at most 32768 and the weights smaller than 4 GiB;
 *   otherwise LB_ESHAPE.  Rows longer than 4096 columns run as column segments of 4096, one launch each on
 *   `s`: the first writes y, each later one adds its partial sums to it (in that fixed order).
 */
lb_status dense_head_matvec(const uint16_t *W, int64_t N, int64_t K, const float *x, float *y, hipStream_t s);

/*
 * The planar product computed by bit-serial popcounts: with q = sum_p t_p bit_p(q) (t_p = 2^p, t_7 = -128),
 * acc = sum_p t_p (popcount(pos & Q_p) - popcount(neg & Q_p)) over the activation bit planes Q_p (tritium
 * "Architecture", section 4.3 "About popcount": the formulation kept as a third independent implementation
 * for differential tests; section 5: the implementations must agree).  Same arguments and output rule as
 * lowbit_matvec for LB_TERNARY_PLANAR with LB_ACT_I8_ROW activations, plus row_sums (device int32 [N],
 * 4-byte aligned, may be NULL): the exact integer acc per row.  y may be NULL when row_sums is not.
 * Results are bit-identical to lowbit_matvec / lowbit_block_sums.  K <= 8192; otherwise LB_ESHAPE.
 */
lb_status lowbit_matvec_popcount(const void *W, int64_t N, int64_t K, float w_tensor_scale, const int8_t *xq,
                                 const float *xscale, float *y, int32_t *row_sums, hipStream_t s);

/*
 * int8 dense head matvec y[n] = row_scale[n] * sum_k W[n][k] * x[k], accumulated in fp32 (tritium
 * "Architecture", section 10: int8 is the obvious move for the head, at half the bf16 head's bytes; the
 * reading taken: symmetric int8 weights with one fp32 scale per row).
 *   W: device int8 [N][K], 16-byte aligned; row_scale: device fp32 [N], 4-byte aligned; x: device fp32 [K],
 *   16-byte aligned; y: device fp32 [N], 4-byte aligned.  K must be a multiple of 16 and at most 32768 and
 *   the weights smaller than 4 GiB; otherwise LB_ESHAPE.  Rows longer than 8192 columns run as column
 *   segments of 8192, one launch each on `s`: the first writes row_scale[n] times its partial sum, each
 *   later one adds its own (in that fixed order).
 */
lb_status dense_head_matvec_i8(const int8_t *W, const float *row_scale, int64_t N, int64_t K, const float *x, float *y,
                               hipStream_t s);

/*
 * Many independent decode products in ONE launch (a token's work list).  A batch is a set-up object:
 * lowbit_batch_create validates the host-side list, and copies it with its tile table into device
 * memory it allocates once; lowbit_matvec_batched then enqueues, on `s`, one kernel per (weight format,
 * kernel configuration) group of the list -- one or two for a model's token -- over every product.
 * (tritium "Architecture", section 7: handing each small matvec to a pool costs more than the matvec
 * itself -- dispatch, not arithmetic, is what a token's many products must amortise.)
 */
typedef struct {
    int32_t fmt;          /* lb_wfmt */
    int32_t afmt;         /* lb_afmt, paired with fmt as in lowbit_matvec */
    int64_t N, K;         /* rows, columns */
    const void *W;        /* device layout, 16-byte aligned */
    float w_tensor_scale; /* planar only */
    const int8_t *xq;     /* device int8 [K] (ignored for LB_ACT_F32_Q8_0) */
    const void *xscale;   /* device binary16 [K/32] or fp32 [1] (ignored for LB_ACT_F32_Q8_0) */
    float *y;             /* device fp32 [N] */
    const float *x;       /* LB_ACT_F32_Q8_0 only: device fp32 [K], 16-byte aligned; else ignored */
} lb_matvec_desc;

typedef struct lb_batch lb_batch;

/* list: HOST array of n descriptors (n >= 1).  On success *out owns device memory until destroyed;
 * lowbit_batch_destroy frees it (hipFree, which waits for the device), so no launch may use it after.
 * The buffers the descriptors point to must stay valid while the batch is used.  A descriptor with
 * afmt LB_ACT_F32_Q8_0 takes its activations from x and needs fmt LB_Q1_0, LB_Q2_0_G64 or LB_Q4_0 (else
 * LB_EUNSUPPORTED); null x is LB_EINVAL, x not 16-byte aligned LB_EALIGN. */
lb_status lowbit_batch_create(const lb_matvec_desc *list, int32_t n, lb_batch **out);
lb_status lowbit_matvec_batched(const lb_batch *b, hipStream_t s);
/* Kernel launches one lowbit_matvec_batched call makes (the quantise launches of long fp32 rows plus one
 * per weight format and kernel configuration present); -1 for a null batch. */
int32_t lowbit_batch_launches(const lb_batch *b);
void lowbit_batch_destroy(lb_batch *b);

/*
 * For callers that cannot allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): the work list of lowbit_batch_create run in one call, with its
 * descriptor and tile tables held in a fixed device array of LB_STATIC_TABLE_BYTES bytes inside the library
 * instead of memory the library allocates.  Calls no hipMalloc / hipFree; the tile plan is built in host
 * memory on every call.
 *   list: HOST array of n descriptors, validated exactly as by lowbit_batch_create (same status codes);
 *         the same products give bit-identical outputs as a batch of that list (here every fp32 row,
 *         however long, is quantised inside its products' launches).
 *   A list whose tables exceed LB_STATIC_TABLE_BYTES (64 bytes per product plus 8 per row tile: for
 *   example 14,000 single-tile products, or 130,000 tiles -- about 8 GB of Q1_0 / Q2_0 weights in their
 *   64 KiB tiles, 32 GB in 256 KiB tiles) is refused with LB_ESHAPE before anything is enqueued.
 * The tables are copied into the array on `s` (stream-ordered after earlier work on `s`), then the kernels
 * run on `s`.  Every call on one GPU shares that GPU's array, which keeps the last call's tables: calls
 * that overlap on one GPU -- on different streams, or from different host threads without ordering --
 * race and may compute with another call's tables.  Calls queued on one stream are safe.
 */
#define LB_STATIC_TABLE_BYTES (1 << 20)
lb_status lowbit_matvec_batched_static(const lb_matvec_desc *list, int32_t n, hipStream_t s);

/*
 * ---- Serving: the steps of a token between and after the products --------------------------------------
 *
 * A batch of B requests holds its keys and values in one paged cache a layer, 4 bits a value.  A step brings
 * new_lens[b] new tokens of request b: lowbit_kv_plan gives them pages and slots, lowbit_kv_append quantises
 * their keys and values into the slots, lowbit_kv_attention lets their queries attend to all of the request, and
 * after the head lowbit_logits_process prepares the logits for sampling.  (The KV cache is the state that the
 * bankml build history's 0.3.9 entry quantises with q8_0; the sampler's penalties, biases and grammars are those
 * of the bankml technical report, section IV.4.)
 *
 * The cache of a layer (lowbit_kv_cache_bytes): `pages` pages of page_tokens tokens P (a power of two, 16 to
 * 1024), a record of P * head_dim * 9 / 8 bytes per page and kv head, [pages][kv_heads][record].  32 consecutive
 * values of a head share a binary16 scale d = fp16_rne(amax * fp32(1/6)) (an fp32 product, at most 65504), and a code
 * is the E2M1 number (sign, then 0 .5 1 1.5 2 3 4 6) nearest to x / d, ties to the even code; all codes are 0
 * where d = 0, and a block with a value that is not finite reads back as NaN.  With nb = head_dim / 32:
 *   K codes  [P][4][nb][4 bytes]     byte (g, b, i): elements 32b + 8g + 2i (lower code) and 32b + 8g + 2i + 1
 *   V codes  [P/4][16][4][nb bytes]  quad of tokens, c, token of the quad, byte i: elements 32i + c, 32i + 16 + c
 *   K scales [P/4][nb][4] binary16   quad of tokens, block, token of the quad; then the V scales alike
 * head_dim is 64, 128 or 256.  A slot is page * P + token of the page, in 64 bits.
 *
 * Rows (queries, keys, values, outputs) are [T][heads][head_dim] of type `dtype` with a stride between tokens in
 * elements (so that they may be parts of wider rows); pointer and stride are multiples of 16 bytes.  What these
 * entry points read on the device (lengths, tables, slots, token numbers) is checked by the kernels: no value of
 * them leads outside the buffers that the sizes describe.
 */
typedef enum { LB_F32 = 0, LB_BF16 = 1, LB_F16 = 2 } lb_dtype;

/* Bytes of one layer's cache; -1 for a bad shape (also one of pages of 4 GiB or more, which nothing here takes). */
int64_t lowbit_kv_cache_bytes(int64_t pages, int64_t kv_heads, int64_t page_tokens, int64_t head_dim);

/*
 * The pages and slots of a step, from the requests' lengths.  Request b holds kv_lens[b] tokens in the pages
 * block_table[b][0 ..] ([B][table_stride]) and brings new_lens[b] >= 0.  Its ceil((len + new) / P) - ceil(len / P)
 * new pages come off the top of the free list: in order of requests and blocks, the i-th new page of the step is
 * free_pages[free_count - 1 - i].  All device int32 (slots int64); written:
 *   block_table        the entries of the new pages (no others)
 *   kv_lens_out [B], free_count_out [1]   lengths and free pages after the step; may be kv_lens, free_count
 *   cu_q [B+1], cu_pages [B+1]            running sums of the new tokens and of the new pages
 *   slots, positions [max_tokens]         of new token i of request b, at cu_q[b] + i: its slot and its place in
 *                                         the request (from 0); behind the last token, slot -1 and position 0
 *   status [3]         0, or a sum of 1: too few free pages, 2: over max_tokens tokens, 4: a negative length, or
 *                      one beyond its table or 2^31 - 1, 8: a free count below 0 or above free_capacity;
 *                      then the pages and the tokens that the step asked for.
 * All or nothing: where status[0] is not 0, no table entry, length or count changes, the sums are 0 and all slots
 * -1, so that the step's other calls do nothing.  B = 0: nothing is read or written, slots included.  At most 2^30
 * requests.  One launch up to 2048 requests and max_tokens 8192, else two.
 */
lb_status lowbit_kv_plan(const int32_t *new_lens, int64_t B, int64_t page_tokens, const int32_t *kv_lens, int32_t *kv_lens_out,
                         int32_t *block_table, int64_t table_stride, const int32_t *free_pages, int64_t free_capacity,
                         const int32_t *free_count, int32_t *free_count_out, int32_t *cu_q, int32_t *cu_pages, int64_t *slots,
                         int32_t *positions, int64_t max_tokens, int32_t *status, hipStream_t s);

/*
 * The pages of the requests with done[b] != 0 go back on top of the free list (in order of requests and blocks),
 * and their lengths become 0.  status [2]: 0, or a sum of 4: a length beyond its table, 8: the list would pass
 * free_capacity, or its count is below 0 (then no length and no count changes); and the pages given back.  Fewer than
 * 2^24 requests.
 */
lb_status lowbit_kv_release(const int32_t *done, int64_t B, int64_t page_tokens, int32_t *kv_lens, const int32_t *block_table,
                            int64_t table_stride, int32_t *free_pages, int64_t free_capacity, int32_t *free_count, int32_t *status,
                            hipStream_t s);

/*
 * Quantises T rows of keys and values into the slots of a layer's cache.  A row whose slot is negative or past
 * the cache is left out.  Two rows with the same slot leave a mixture of both there.  T * kv_heads * head_dim below
 * about 2^35 (here and in lowbit_kv_read).
 */
lb_status lowbit_kv_append(int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int64_t T, int64_t kv_heads,
                           int64_t head_dim, const int64_t *slots, void *cache, int64_t pages, int64_t page_tokens, hipStream_t s);

/* The rows of T slots as the cache holds them (code times scale, rounded to dtype); zeros for a slot outside. */
lb_status lowbit_kv_read(int dtype, const void *cache, int64_t pages, int64_t page_tokens, int64_t T, int64_t kv_heads, int64_t head_dim,
                         const int64_t *slots, void *k, int64_t k_stride, void *v, int64_t v_stride, hipStream_t s);

/*
 * lowbit_kv_append of keys turned by their positions, and the step's queries turned alike, in one pass.  Row t stands at
 * positions[t] (int32; lowbit_kv_plan writes them).  Of every head, the first rotary_dim elements (a multiple of 16, at
 * least 16, at most head_dim) are rotary_dim / 2 pairs (x, y), and the rest stay as they are:
 *   LB_ROTARY_HALVES  pair i: elements i and i + rotary_dim / 2;    LB_ROTARY_PAIRS  pair i: elements 2i and 2i + 1
 *   a = positions[t] * inv_freq[i],  (x, y) -> factor * (x cos a - y sin a,  y cos a + x sin a)
 * inv_freq: device fp32 [rotary_dim / 2]; whatever scaling of long contexts a model has is in them and in factor.
 * Angles, sines and products are in 64 bits; a turned element is rounded to fp32 and then to dtype.  The cache's bytes are
 * those of turning first and lowbit_kv_append.  q_out may be q, with the same stride, but not overlap it otherwise, nor k, v;
 * q_heads may be 0 (q and q_out are not used then).  A row whose slot is negative or past the cache is left out: neither
 * cache nor q_out change.  T * (q_heads + kv_heads) * head_dim below about 2^35, and at most 65535 heads in all.
 */
typedef enum { LB_ROTARY_HALVES = 0, LB_ROTARY_PAIRS = 1 } lb_rotary;
lb_status lowbit_kv_append_rotary(int dtype, const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, const void *k,
                                  int64_t k_stride, const void *v, int64_t v_stride, int64_t T, int64_t q_heads, int64_t kv_heads,
                                  int64_t head_dim, const int32_t *positions, const float *inv_freq, int64_t rotary_dim, int style,
                                  float factor, const int64_t *slots, void *cache, int64_t pages, int64_t page_tokens, hipStream_t s);

/*
 * Causal attention of a step's new tokens.  Request b's queries are rows cu_q[b] .. cu_q[b+1] - 1 of q and out
 * (at most max_q of them, T rows in all), the last tokens of its kv_lens[b] <= max_kv tokens (new ones included,
 * already appended), found through block_table[b].  Query i of n, at position pos = kv_lens[b] - n + i, sees the
 * keys j with j <= pos, and with window > 0 only those with j > pos - window:
 *   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q . k_j - max),  head h reading kv head h / (q_heads / kv_heads).
 * A query that sees no key (kv_lens[b] < n) gives zeros; rows before the first request's (cu_q[0] of them) and behind
 * the last's are left as they were.  A page number outside the cache, among those that a query sees, makes the
 * query's result NaN, as does a request longer than max_kv or than its table.  A request of more than max_q tokens may
 * leave rows unwritten.
 * out may be q, with the same stride, but not overlap it otherwise.
 * Precision: sums, maxima and exponents are 32-bit, the result is rounded to dtype once.  Scores (scale * q . k) are
 * taken up to 2^24 in size; beyond, where fp32 no longer tells neighbours apart, a result may not be finite.  On the
 * way, in relative terms and for what is far below its row's largest in terms of that:
 *   queries  fp32 2^-22, the others exact; 2^-39 of the row's largest element
 *   weights  p_j times the value's scale: fp32 2^-21, the others 2^-11; 6 * 2^-31 a key of the largest such product (a
 *            scale of 0 counted as 2^-64): of the element's own 32-block where requests have at most 512 / head_dim
 *            rows (max_q times q_heads / kv_heads), else of all blocks.  So fp32 elements are good to 2^-20 of
 *            sum_j p_j |v_j| where their block's values are not below some 2^-10 of the row's largest.
 *   and for 16-bit rows where requests may have over 64: p_j alone, 2^-11 and 2^-31 of the largest; and the keys and
 *            values (code times scale), 2^-11 and 2^-30 of the largest scale among the request's keys, or values.
 * workspace: lowbit_kv_attention_workspace(...) bytes, 16-byte aligned, for the joining of long requests' parts
 * (0 bytes, NULL, where none are split); calls that may run at the same time need one each.
 * Limits (LB_ESHAPE beyond them; the workspace call answers -1 where no row type is left): B and T * q_heads at most
 * 2^31 - 1, and fewer than 2^23 tiles, or parts of split ones.  A kv head has a tile for every 16 rows (query token
 * and head of its group), and one more a request; for 16-bit rows, where requests may have over 64, every 128 or 256:
 * T * q_heads below about 2^27 for fp32 rows, and all of 2^31 for the others where B is small.
 */
int64_t lowbit_kv_attention_workspace(int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_q,
                                      int64_t max_kv, int64_t window);
lb_status lowbit_kv_attention(int dtype, const void *q, int64_t q_stride, int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads,
                              int64_t head_dim, const int32_t *cu_q, const int32_t *kv_lens, const int32_t *block_table,
                              int64_t table_stride, const void *cache, int64_t pages, int64_t page_tokens, int64_t max_q,
                              int64_t max_kv, float scale, int64_t window, void *out, int64_t out_stride, void *workspace,
                              int64_t workspace_bytes, hipStream_t s);

/*
 * Routing of T tokens to E experts (1 to 1024).  logits [T][E] of type dtype, row stride `stride` elements.  Per token:
 *   scores   p = softmax over the E logits (LB_SCORE_SOFTMAX), or 1 / (1 + exp(-logit)) (LB_SCORE_SIGMOID)
 *   order    experts by p + bias[e] (bias: device fp32 [E], NULL for none), the largest first, equal ones by index
 *   groups   of E / groups experts each (1 to 64 of them): only the groups_kept groups with the largest sums of their
 *            group_best (1 or 2) largest values p + bias are looked at; equal ones by index
 *   chosen   the first top_k (1 to 64): experts[t][j], in order; their weights are p, without the bias, over the sum of the
 *            top_k where renormalise is not 0 (0 where that is 0), times factor: weights[t][j]
 * Scores, sums and comparisons are in 64 bits, weights rounded to fp32 once.  A NaN logit counts as -inf, and a softmax of
 * logits of -inf alone is that of equal ones; of infinite ones, those share it; a p + bias that is NaN or -inf comes last.
 * count: device int32, NULL for T; tokens from count[0] on (a padded step's; the last of lowbit_kv_plan's cu_q is that
 * number) get experts -1 and weights 0.  T below 2^26, and at most 2^26 - 4 with more than 256 experts or 32 groups.
 */
typedef enum { LB_SCORE_SOFTMAX = 0, LB_SCORE_SIGMOID = 1 } lb_score;
lb_status lowbit_route(int dtype, const void *logits, int64_t stride, int64_t T, int64_t E, int score, const float *bias, int64_t groups,
                       int64_t groups_kept, int64_t group_best, int64_t top_k, int renormalise, float factor, const int32_t *count,
                       int32_t *experts, float *weights, hipStream_t s);

/*
 * The products of the routed pairs.  The experts' N x K tensors lie one after another, each lowbit_pack_weights' layout
 * padded to a multiple of 16 bytes: lowbit_experts_weight_bytes(fmt, 1, N, K) from one to the next (-1 for a bad shape, or
 * a tensor of 4 GiB or more).
 *
 * lowbit_experts_plan sorts `pairs` pairs by expert (experts: device int32 [pairs]; a number outside 0 .. E-1 is a pair
 * that is left out, as a padded token's -1) into `plan` (device, lowbit_experts_plan_bytes(pairs, E) bytes, 16-byte
 * aligned), for any number of products of the same pairs and E.  The order does not depend on how anything runs.  At most
 * 2^30 pairs and 1024 experts.
 */
int64_t lowbit_experts_weight_bytes(int fmt, int64_t E, int64_t N, int64_t K);
int64_t lowbit_experts_plan_bytes(int64_t pairs, int64_t E);
lb_status lowbit_experts_plan(const int32_t *experts, int64_t pairs, int64_t E, void *plan, hipStream_t s);

/*
 * y[p] = W[experts[p]] . dequant(x[p / pairs_per_row]) for every pair p that is not left out (y's other rows are not
 * written): pairs_per_row is top_k where a token's pairs share its activations (an expert's first products), 1 where each
 * pair has its own (its last).  fmt LB_Q1_0, LB_Q2_0_G64 or LB_Q4_0 (others LB_EUNSUPPORTED); xq int8
 * [ceil(pairs / pairs_per_row)][K] and xscale binary16 [..][K/32] are q8_0 rows (lowbit_quantize_act); y fp32 [pairs][N].
 * With a plan, weights are read once for up to 16 or 128 rows, and `experts` is not read; without (NULL), each pair is
 * computed by itself, with lowbit_matvec's results, which is best for a single token and up to about half a pair an
 * expert.  Integer block sums are exact and scaled as lowbit_matvec does, in an order that depends on
 * the sizes and on how many pairs an expert has.
 * Limits: K a multiple of 128 (64 for LB_Q2_0_G64), at most 32768 (16384 for LB_Q4_0); xq below 4 GiB.
 */
lb_status lowbit_experts_matmul(int fmt, const void *W, int64_t E, int64_t N, int64_t K, const int8_t *xq, const void *xscale,
                                const int32_t *experts, int64_t pairs, int64_t pairs_per_row, const void *plan, float *y, hipStream_t s);

/*
 * out[t] = sum over j of weights[t][j] * y[t * top_k + j], for the pairs with an expert in 0 .. E-1 (the others' rows are not
 * read; a token without any gives zeros).  y fp32 [T * top_k][N], out [T][N] of type dtype with a stride in elements.
 * Summed in fp32 in the order of j, rounded once.  out must not overlap y.  T * N below about 2^32.
 */
lb_status lowbit_experts_combine(int dtype, const float *y, const int32_t *experts, const float *weights, int64_t T, int64_t top_k, int64_t E,
                                 int64_t N, void *out, int64_t out_stride, hipStream_t s);

/*
 * Logits before sampling: logits [B][V] of type `dtype`, row stride in_stride elements; out alike (it may be
 * logits itself, with the same stride, but not overlap it otherwise).  In fp32, for every token t of row b, in
 * this order, rounded to dtype once at the end:
 *   penalties  t anywhere in the history tokens[b][0 .. total_lens[b]): l = l > 0 ? l / repetition[b] : l * repetition[b];
 *              t count times in its output part, from prompt_lens[b] on, count > 0: l -= frequency[b] * count, then
 *              l -= presence[b]
 *   biases     l += the sum of the values of t's entries in bias_tokens[b][0 .. bias_lens[b]), added in list order
 *   mask       l = -inf where bit t % 32 of mask[b][t / 32] is 0
 * tokens, repetition, presence, frequency, bias_tokens and mask may be NULL (left out), prompt_lens too (all of the
 * history is output).  Lengths are cut to the strides; token numbers outside 0 .. V-1 are passed over.  At most
 * 16384 biases a row, and B * ceil(V / 1024) below 2^22.  Results do not depend on the order in which anything runs.
 */
lb_status lowbit_logits_process(int dtype, const void *logits, int64_t in_stride, int64_t B, int64_t V, const int32_t *tokens,
                                int64_t tok_stride, const int32_t *prompt_lens, const int32_t *total_lens, const float *repetition,
                                const float *presence, const float *frequency, const int32_t *bias_tokens, const float *bias_values,
                                int64_t bias_stride, const int32_t *bias_lens, const uint32_t *mask, int64_t mask_stride, void *out,
                                int64_t out_stride, hipStream_t s);

/*
 * Measurement helper, not a product: a streaming read of `nbytes` (a multiple of 16, 16-byte aligned) of
 * device memory by 16-byte non-temporal loads, the access pattern of the decode kernels' weight stream,
 * so its rate bounds theirs (tritium "Architecture", section 3: the roofline is measured with a
 * streaming-read probe in the same run).  `sink` (device uint32, at least 65536 entries, 4-byte aligned) is
 * written only when a workgroup's checksum of the bytes equals a fixed constant, so the loads cannot be
 * removed and almost nothing is written.
 */
lb_status lowbit_read_probe(const void *buf, int64_t nbytes, uint32_t *sink, hipStream_t s);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_H */

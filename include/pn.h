/*
 * pn.h -- C ABI of libpn.so: decode-step GEMV y = W.x over block-quantized weights decoded in
 * registers, and a step's key/value cache, attention and verification of drafts, on AMD Instinct
 * MI355X (gfx950).
 *
 * Formats:
 *   PN (pn3t, pn4t)  "PN weight format" (PNX-FORMAT-v0), sections "Types", "Block layout",
 *                    "Value", "Reference quantizer", "Validation".
 *   NVFP4 (W4A16)    "Quantisation and profiles", sections "NVFP4" and "The clip search";
 *                    NInfer "tensor formats", section 3.3 (E2M1 and E4M3FN words, validity).
 *   row-scaled E4M3  NInfer "tensor formats", section 3.4 (FP8_E4M3FN_ROW_BF16S);
 *                    "Quantisation and profiles", "The FP8 head".
 *
 * Conventions for every entry point:
 *   - Every pointer argument that names a tensor is a DEVICE pointer, owned by the caller. The
 *     library allocates nothing and keeps no pointer after the call returns.
 *   - `stream` is a hipStream_t (NULL = the default stream). Work is enqueued asynchronously on it;
 *     the call returns after argument checks and kernel launch, not after completion.
 *   - The return value is a status (PN_OK = 0, or a negative PN_ERR_*), decided synchronously from
 *     the arguments and the launch. Per-row verdicts and quantizer statuses are device outputs.
 *   - Nothing falls back silently: a shape, dtype or device this library does not handle is an
 *     error, never a slower path on another device.
 *   - N == 0, nrows == 0 or M == 0 is a no-op that returns PN_OK. K must be a positive whole
 *     number of blocks (80 for pn3t, 64 for pn4t, 16 for NVFP4); otherwise PN_ERR_SHAPE.
 *
 * PN tensor layout: W is N rows of K weights; row n starts at byte n * pn_row_bytes(type, K); a
 * row is K/80 (pn3t) or K/64 (pn4t) consecutive 34-byte blocks. Block b of a row starts at byte
 * 34*b: bytes 0..1 hold d (fp16, little-endian, signed), bytes 2..33 hold eight little-endian u32
 * words. W needs only 2-byte alignment; nothing assumes a word is 4-byte aligned.
 */
#ifndef PN_H
#define PN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ggml type ids of the two PN types ("PN weight format", "Types"). */
enum { PN_TYPE_PN3T = 124, PN_TYPE_PN4T = 125 };

/* Status codes. */
enum {
    PN_OK = 0,
    PN_ERR_TYPE = -1,   /* type is neither PN_TYPE_PN3T nor PN_TYPE_PN4T */
    PN_ERR_SHAPE = -2,  /* K is not a positive whole number of blocks, or a size is negative */
    PN_ERR_TOKENS = -3, /* M (tokens) outside 0..16 (PN GEMV) or 0..4 (NVFP4, row-scaled E4M3) */
    PN_ERR_NULL = -4,   /* a required pointer is NULL */
    PN_ERR_ALIGN = -5,  /* W not 2-byte aligned, x / y / w not 4-byte aligned, bf16 x not 2-byte,
                           NVFP4 codes not 8-byte aligned */
    PN_ERR_HIP = -6,    /* the HIP runtime reported an error (no device, launch failure) */
    PN_ERR_DEVICE = -7, /* the current device is not gfx950 */
    PN_ERR_HADAMARD = -8, /* Hadamard slice size B is not a power of two in 2..16384 dividing K */
    PN_ERR_FORMAT = -9,   /* unknown cache format or element type */
    PN_ERR_WORKSPACE = -10 /* the workspace is smaller than the call needs */
};

/* Maximum tokens per GEMV call. */
#define PN_MAX_TOKENS 4        /* NVFP4 and row-scaled E4M3 GEMV */
#define PN_GEMV_MAX_TOKENS 16  /* PN GEMV */
#define PN_GEMV_GROUP_MAX_PARTS 4  /* matrices per pn_gemv_group call */
#define PN_GEMV_HADAMARD_MAX_TOKENS 4  /* PN GEMV with the rotation fused */

/* Bytes of one PN row of K weights: 34*K/80 (pn3t) or 34*K/64 (pn4t); 0 if K is not a positive
 * multiple of the block size or type is unknown. Host-only, no device work. */
int64_t pn_row_bytes(int type, int64_t K);

/* Human-readable name of a status code (static storage). */
const char *pn_status_string(int status);

/* ---- PN validation ("PN weight format", "Validation") --------------------------------------
 * verdict[r] = 1 if row r is valid, 0 if it is invalid: some block's d is an fp16 NaN or infinity,
 * or (pn3t) bit 15 or bit 31 of some word is set. verdict is int32[nrows] on the device. */
int pn_validate_rows(int type, const void *W, int64_t nrows, int64_t K, int32_t *verdict,
                     void *stream);
/* One row (nrows = 1). */
int pn_validate_row(int type, const void *row, int64_t K, int32_t *verdict, void *stream);

/* ---- PN decode ("PN weight format", "Value") -----------------------------------------------
 * out[r*K + k] = fp32(d) * (n - z) for every weight, bit-exact: the product is exact in fp32, IEEE
 * signs apply (code z with a negative d gives -0.0; d = +0 with n < z gives -0.0), fp16 subnormal
 * d are kept. Reserved bits are ignored by the decode (they only make the row invalid). A
 * non-finite d decodes as the IEEE product (NaN or +-inf). out is fp32[nrows, K]. */
int pn_dequantize_rows(int type, const void *W, int64_t nrows, int64_t K, float *out,
                       void *stream);
int pn_dequantize_row(int type, const void *row, int64_t K, float *out, void *stream);

/* ---- PN GEMV -------------------------------------------------------------------------------
 * y[m*N + n] = sum_k w[n, k] * x[m*K + k] for m < M (1 <= M <= 16 tokens), with w the decode above,
 * accumulated in fp32. x is fp32[M, K] row-major, y fp32[M, N] row-major (overwritten).
 * Accuracy ("PN weight format", "Value"): |y - y_ref| <= 1e-5 * sum_k |w_k x_k| per output, y_ref
 * the exact sum, for every finite input whose products and partial sums stay in fp32's normal
 * range. At 1-4 tokens each weight is decoded exactly to the integer n - z, each product with x is
 * exact inside an fp32 fma, and the only roundings are the fp32 sums: eight chains of at most 10
 * terms per lane and block piece, one multiply by d, a 64-lane tree and the in-order sum of at most
 * a few dozen chunk partials per row (under 30 * 2^-24 of sum_k |w x| in the worst case).
 * At 5-16 tokens (the matrix cores) the zero point is taken off each code exactly as well, but
 * each x is carried as an fp16 (hi, lo) pair with one exponent per token and group of blocks (4
 * consecutive blocks where W is staged through LDS, one block where it is read directly): exact to
 * 2^-22 relative or to 2^-32 (pn3t; 2^-34 pn4t) of the largest |x| in its group, whichever is
 * larger, so the bound above holds where every x that meets a nonzero weight is within about 2^14
 * of the largest |x| of its group, or the group's other terms dominate. Rows are not
 * validated here (validate at load); an invalid row gives an unspecified value but no
 * out-of-bounds access. Deterministic: the same inputs and launch give the same bits on every
 * call. */
int pn_gemv(int type, const void *W, int64_t N, int64_t K, const float *x, int64_t M, float *y,
            void *stream);

/* Several PN GEMVs that read the same x (a layer's q, k and v; gate and up):
 * parts[i].y[m*N_i + n] = sum_k w_i[n, k] * x[m*K + k], with the bits of one pn_gemv per part. At
 * 1-4 tokens all parts, of either type, run as one launch where the shapes allow it (else the
 * parts of each type, else one launch per part, in order on the stream). 1 <= count <=
 * PN_GEMV_GROUP_MAX_PARTS (else PN_ERR_SHAPE); every part has its own type, W (N_i rows of K
 * weights) and y, and all share K, x and M (0..16). Argument errors as pn_gemv, for the first part
 * that has one; parts with N = 0 are skipped. The parts' y must not overlap each other or x. */
typedef struct pn_gemv_part {
    int type;       /* PN_TYPE_PN3T or PN_TYPE_PN4T */
    const void *W;  /* N rows of pn_row_bytes(type, K) bytes, 2-byte aligned */
    int64_t N;      /* rows (outputs per token) */
    float *y;       /* fp32[M, N], 4-byte aligned */
} pn_gemv_part;
int pn_gemv_group(const pn_gemv_part *parts, int count, int64_t K, const float *x, int64_t M,
                  void *stream);

/* ---- Hadamard-rotated activations ("PN weight format", "Files that use PN") ----------------
 * The page states that the model rotates the activations that reach the PN weights with a
 * Hadamard transform, done by the engine, and fixes neither its order nor its normalisation.
 * Reading used here: each row of x[M, K] is cut into consecutive slices of B elements (B a power
 * of two, 2 <= B <= 16384, dividing K; otherwise PN_ERR_HADAMARD), and each slice is multiplied by
 * the orthonormal Sylvester-ordered Walsh-Hadamard matrix H_B / sqrt(B),
 * H_B[i][j] = (-1)^popcount(i & j):  x'[m, s*B + i] = sum_j H_B[i][j] x[m, s*B + j] / sqrt(B).
 * Computed in fp32 as log2(B) butterfly stages and one multiply by fp32(1/sqrt B) (exact for even
 * log2 B): |x' - x'_exact| <= (log2(B) + 2) * 2^-24 * sum_j |x[m, s*B + j]| / sqrt(B) per element
 * (up to terms in 2^-48). Deterministic. */

/* out[M, K] = the rotation of x[M, K] (fp32, row-major). K must be a multiple of 4
 * (PN_ERR_SHAPE). out may equal x (in place); otherwise they must not overlap. */
int pn_hadamard_rows(const float *x, int64_t M, int64_t K, int64_t B, float *out, void *stream);

/* y = W x' for M = 1..4 tokens: the rotation of pn_hadamard_rows into a workspace, then pn_gemv
 * on it: the same bits as those two calls made by hand, the rotation's error above adding to the
 * GEMV's; x itself is not modified. The workspace is a buffer per stream (up to 16 streams per
 * device) that the library keeps for the life of the process, grown on its stream
 * (hipMallocAsync, the old one hipFreeAsync'd) when a call needs more than it holds: a call
 * allocates nothing otherwise. Calls on one stream reuse its buffer in stream order; calls on
 * different streams never share one. Past 16 streams on a device, on hipStreamPerThread and under
 * stream capture, a call takes a temporary instead (hipMallocAsync and hipFreeAsync on its stream,
 * which a graph records as nodes of its own). Arguments as pn_gemv, plus B as in
 * pn_hadamard_rows; M outside 0..4 gives PN_ERR_TOKENS, a failed allocation PN_ERR_HIP. */
int pn_gemv_hadamard(int type, const void *W, int64_t N, int64_t K, const float *x, int64_t M,
                     int64_t B, float *y, void *stream);

/* pn_gemv_hadamard without any allocation, for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid it). The rotated x goes to a
 * file-scope device array of PN_NOALLOC_MAX_FLOATS floats (1 MiB) that each GPU holds for the life
 * of the process; the rotation overwrites every element the GEMV then reads, so nothing is cleared
 * between calls. Same arguments, errors and bits as pn_gemv_hadamard, plus PN_ERR_SHAPE when
 * M * K exceeds PN_NOALLOC_MAX_FLOATS. Every call on one GPU shares that GPU's array: calls that
 * overlap on one GPU (on different streams, or from several host threads) race on it, so callers
 * order them. */
#define PN_NOALLOC_MAX_FLOATS 262144
int pn_gemv_hadamard_noalloc(int type, const void *W, int64_t N, int64_t K, const float *x,
                             int64_t M, int64_t B, float *y, void *stream);

/* Several GEMVs that share x, over the rotated x: x rotated once into the workspace of
 * pn_gemv_hadamard (same streams and allocation), then pn_gemv_group on it -- parts[i].y = W_i x'
 * with the bits of pn_hadamard_rows followed by one pn_gemv per part. B as in pn_hadamard_rows,
 * 0 <= M <= 4 (else PN_ERR_TOKENS), parts and errors as pn_gemv_group. */
int pn_gemv_group_hadamard(const pn_gemv_part *parts, int count, int64_t K, const float *x,
                           int64_t M, int64_t B, void *stream);

/* ---- PN reference quantizer ("PN weight format", "Reference quantizer") ---------------------
 * Quantizes fp32 w[nrows, K] (row-major) into PN rows W (nrows * pn_row_bytes bytes), one group of
 * 80 or 64 weights per block: 36 candidate scales s = fp16(sigma * m * amax / z),
 * m = 0.50, 0.52, ..., 1.20, codes clamp(rint(w/s) + z, 0, 2z-1), double-precision squared error,
 * ties to the larger m; an all-zero group, or one whose candidates all round to zero, is the
 * canonical zero group (d = +0, codes z). Every step runs in fp64 in the order stated, so these
 * rules fix every output bit.
 * status (int32[nrows], optional, may be NULL) receives per row the OR of: 1 = a group held a NaN
 * or infinity, 2 = every candidate scale overflowed fp16 (such groups are written as the canonical
 * zero group). */
int pn_quantize_rows(int type, const float *w, int64_t nrows, int64_t K, void *W, int32_t *status,
                     void *stream);

/* ---- NVFP4 W4A16 ---------------------------------------------------------------------------
 * Layout: codes uint8[N, K/2], element k of a row in byte k/2, even k in the low nibble (E2M1
 * words); scales uint8[N, K/16], one E4M3FN word per group of 16 consecutive k; one fp32 global
 * multiplier g (weight_scale_2). A weight is fp32(fp32(e2m1(code) * e4m3(scale)) * g). */

/* verdict[n] = 1 iff every scale word of row n has sign bit 0 and is not NaN (0x7F), and g is
 * finite and > 0. */
int pn_nvfp4_validate_rows(const uint8_t *scales, float g, int64_t N, int64_t K, int32_t *verdict,
                           void *stream);

/* out fp32[N, K], bit-exact decode as above. */
int pn_nvfp4_dequantize_rows(const uint8_t *codes, const uint8_t *scales, float g, int64_t N,
                             int64_t K, float *out, void *stream);

/* y[m*N + n] = sum_k w[n, k] * x[m, k], x bf16[M, K] (raw 16-bit words, row-major), 1 <= M <= 4,
 * fp32 accumulation; same accuracy contract as pn_gemv. codes must be 8-byte aligned (rows of
 * K/2 bytes with K a multiple of 16 keep every row 8-byte aligned), else PN_ERR_ALIGN. */
int pn_gemv_nvfp4(const uint8_t *codes, const uint8_t *scales, float g, int64_t N, int64_t K,
                  const uint16_t *x_bf16, int64_t M, float *y, void *stream);

/* ---- Row-scaled E4M3FN (FP8_E4M3FN_ROW_BF16S) -----------------------------------------------
 * NInfer "tensor formats", section 3.4: codes uint8[N, K] E4M3FN words (section 3.3), row-major;
 * one bfloat16 multiplier word per row, scales uint16[N]; w = binary32(e4m3(c) * bf16(s)).
 * "Quantisation and profiles", "The FP8 head": the output head (248,320 x 5,120) is stored this
 * way, one scale per vocabulary row. */

/* verdict[n] = 1 iff row n is valid: its multiplier has sign bit 0 and is finite (+0 and positive
 * subnormals included), no code is a NaN word (0x7F, 0xFF), and a +0 multiplier has only
 * signed-zero codes (0x00, 0x80). */
int pn_fp8row_validate_rows(const uint8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                            int32_t *verdict, void *stream);

/* out fp32[N, K] = binary32(e4m3(code) * bf16(scale)), bit-exact (NaN words decode to NaN). */
int pn_fp8row_dequantize_rows(const uint8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                              float *out, void *stream);

/* y[m*N + n] = sum_k w[n, k] * x[m*K + k], x fp32[M, K], y fp32[M, N] (overwritten), 1 <= M <= 4,
 * fp32 accumulation, |y - y_exact| <= 1e-5 * sum_k |w x| for finite inputs. K must be a multiple of
 * 16 (PN_ERR_SHAPE) and codes 16-byte aligned (PN_ERR_ALIGN). Rows are not validated here.
 * Deterministic. */
int pn_gemv_fp8row(const uint8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                   const float *x, int64_t M, float *y, void *stream);

/* ---- Microscaled key/value cache ---------------------------------------------------------------
 * A paged cache of a layer's keys and values in microscaled floating point, quantised as it is
 * written and decoded in registers as it is read. Per token and KV head, K and V are `dim` channels
 * each (64, 128 or 256) in blocks of 32 channels; a block has one exponent byte b (E8M0) and 32
 * codes of the format's element type:
 *   PN_CACHE_MXFP8  E4M3FN codes, largest magnitude 448
 *   PN_CACHE_MXFP4  E2M1 codes, largest magnitude 6, the even channel in the low nibble
 * A channel stands for element(code) * 2^(b - 127), b = 255 for NaN whatever the code. Writing takes
 * the smallest b >= 16 at which the block's largest magnitude is at most that of the element type
 * times 2^(b - 127), and rounds x * 2^(127 - b), which is exact, once, to the nearest code, ties to
 * the even one, the sign kept: every bit of the cache is fixed by these rules. (b >= 16 keeps every
 * number a normal bfloat16 one.)
 * A block with a NaN, an infinity or a magnitude of 2^127 or more has b = 255 and zero codes.
 *
 * Layout: [pages][heads][page / 32] records of 32 tokens, each of pn_cache_page_bytes / (heads *
 * page / 32) bytes: K codes, V codes, K exponents, V exponents. In a record, with token 16a + i or
 * 16a + 4g + t, channel chunk p of 64, block 2p + h:
 *   K codes      MXFP8 [p][a][g][i][16 channels from 64p + 16g]
 *                MXFP4 [p][g][i][a][16 channels from 64p + 16g]
 *   V codes      MXFP8 [p][a][g][i][t][4 channels from 64p + 4i]
 *                MXFP4 [p][g][i][a][t][4 channels from 64p + 4i]
 *   K exponents  [h][i][p][a]        V exponents  [h][g][p][a][t]
 * which is the order in which the matrix instructions of pn_attend take them: a wave reads each
 * record as one contiguous run. data must be 16-byte aligned (PN_ERR_ALIGN). */
enum { PN_CACHE_MXFP8 = 0, PN_CACHE_MXFP4 = 1 };
/* Element types of plain tensors. */
enum { PN_F32 = 0, PN_BF16 = 1, PN_F16 = 2 };

typedef struct pn_cache {
    int format;    /* PN_CACHE_MXFP8 or PN_CACHE_MXFP4 (else PN_ERR_FORMAT) */
    int heads;     /* KV heads, at least 1 */
    int dim;       /* channels a head: 64, 128 or 256 (else PN_ERR_SHAPE) */
    int page;      /* tokens a page: a power of two in 32..1024 (else PN_ERR_SHAPE) */
    int64_t pages; /* pages in data */
    void *data;    /* pages * pn_cache_page_bytes bytes on the device */
} pn_cache;

/* Bytes of one page; 0 where the format, heads, dim or page is not one of the above. Host-only. */
int64_t pn_cache_page_bytes(int format, int heads, int dim, int page);

/* Quantises T tokens' keys and values into the cache. k and v are of `type`, the channels of a head
 * contiguous, token t and head h at element t * token_stride + h * head_stride. slots int64[T] on
 * the device: token t goes to place slots[t] % page of page slots[t] / page; a slot outside
 * 0 .. pages * page - 1 (a padding token's -1) writes nothing. Slots of one call must differ. k and
 * v need only their element's alignment (4 elements' alignment of bases and strides is faster). */
int pn_cache_write(const pn_cache *cache, int type, const void *k, int64_t k_token_stride,
                   int64_t k_head_stride, const void *v, int64_t v_token_stride,
                   int64_t v_head_stride, const int64_t *slots, int64_t T, void *stream);

/* Reads T tokens back: k and v [T][heads][dim] of `type`, contiguous, aligned to 4 elements: the
 * numbers above, exact in fp32 and bf16, rounded once to fp16. A slot outside the cache gives
 * zeros. Slots may repeat. */
int pn_cache_read(const pn_cache *cache, int type, const int64_t *slots, int64_t T, void *k, void *v,
                  void *stream);

/* ---- Attention over the cache --------------------------------------------------------------------
 * B sequences of Q query tokens each (the tokens of one step: 1, or 1 + the drafted ones) attend to
 * a prefix that all of them share and to their own tokens, both read from the cache (the own tokens
 * include the step's, written before the call). Query token i of sequence b, head hq of Hq (KV head
 * hq / (Hq / heads)):
 *   out = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q.k_j),   lse = log sum_j w_j
 * over every prefix token and the own tokens j <= lens[b] - nq + i, nq = q_lens[b] (Q where q_lens
 * is NULL). A row that sees nothing, and every row i >= nq, is zeros with lse = -infinity; so is one
 * whose every score is -infinity (an infinite q). A score of +infinity or NaN makes the row NaN.
 * The prefix is computed for all sequences at once: its cache is read once per block of rows of all
 * sequences (64 rows, or 128 to 384 by dim and type where there are more), not once per sequence.
 *   q      [B][Q][Hq][dim] of `type` with strides in elements (channels contiguous)
 *   table  int32[B][table_width] (row stride table_stride), the own pages of each sequence;
 *          lens int32[B] own tokens, taken as 0..table_width * page
 *   prefix_table int32[ceil(prefix_len / page)]
 *   out    [B][Q][Hq][dim] of `type`, contiguous, 16-byte aligned; lse fp32[B][Q][Hq] or NULL
 * A page number outside the cache is taken as the nearest one inside it: an unspecified value,
 * no access out of bounds. Tokens past a sequence's length are not used, whatever lies there.
 * Arithmetic: products on the matrix cores with fp32 sums; cache numbers enter exactly (bf16 holds
 * them); maxima and sums in fp32. q enters exactly, fp16 as two bf16 parts and fp32 as three. The
 * softmax weights meet v as three parts for fp32 q (2^-24 relative at most) and as two (2^-16) for
 * fp16 and bf16 q; a prefix under more than 64 rows of a KV head (B * Q * Hq / heads) takes those of
 * bf16 q rounded to bf16 once (2^-8). An output is rounded to its type once. Weights are held relative
 * to a number near their row's largest, at which they may reach 2^12: sums of values past some 2^100
 * can leave fp32 where their mean would not.
 * Deterministic: a row's value depends on the call's shapes and its own data only.
 * workspace: pn_attend_workspace_bytes of device memory (16-byte aligned), overwritten; it may be
 * used by the next call on the same stream, calls that may overlap need one each. */
typedef struct pn_attend_args {
    int type;                 /* PN_F32, PN_BF16 or PN_F16 */
    int B, Q, Hq;             /* Hq a multiple of cache->heads (else PN_ERR_SHAPE) */
    const void *q;
    int64_t q_seq_stride, q_token_stride, q_head_stride;
    float scale;              /* finite */
    const int32_t *table;
    int64_t table_stride;
    int table_width;          /* pages a row of table has, 0 or more */
    const int32_t *lens;
    const int32_t *q_lens;    /* may be NULL */
    const int32_t *prefix_table;
    int64_t prefix_len;
    void *out;
    float *lse;               /* may be NULL */
} pn_attend_args;

/* Device bytes that pn_attend needs for these sizes (0 where none, or a size is invalid). Reads
 * type, B, Q, Hq, table_width and prefix_len of a. */
int64_t pn_attend_workspace_bytes(const pn_cache *cache, const pn_attend_args *a);

int pn_attend(const pn_cache *cache, const pn_attend_args *a, void *workspace,
              int64_t workspace_bytes, void *stream);

/* ---- Verification of drafted tokens --------------------------------------------------------------
 * B sequences with K drafted tokens each (n = n_draft[b] of them, K where n_draft is NULL). p are the
 * target's probabilities at the K + 1 positions, q the draft's at the K positions that the tokens
 * were drawn from, or NULL where each draft is certain (q = 1 at the token, 0 elsewhere).
 * Draft i is accepted iff every earlier one was and u_accept[b][i] * q_i(x_i) < p_i(x_i). After a
 * accepted drafts comes one more token: the smallest t at which r_0 + .. + r_t > u_sample[b] * R,
 * R the sum of all r; r = max(p_a - q_a, 0), where a < n and that has a positive sum, else r = p_a.
 * With u uniform in [0, 1) the tokens are distributed as the target's.
 * Every product, difference, sum and comparison is in 64 bits. A draft whose p or q is NaN or
 * negative is refused, and a token whose p_a or q_a is has r_t = 0 (where r = p_a, p_a alone counts);
 * a draft outside 0..V-1 is refused (and r = p_a where q is NULL). Where no t qualifies (rounding of
 * the last sum, u >= 1) the token is the last t with r_t > 0, and -1 where r is zero everywhere.
 *   p  row (b, i) at element (b * (K + 1) + i) * p_stride, q at (b * K + i) * q_stride, both of
 *      `type`; draft int32[B][K]; u_accept fp32[B][K]; u_sample fp32[B]; n_draft int32[B] or NULL,
 *      taken as 0..K
 *   tokens int32[B][K + 1]: the accepted drafts, the token after them, then -1; accepted int32[B]
 * 0 <= K <= PN_VERIFY_MAX_DRAFTS, 1 <= V < 2^30. Deterministic. The workspace is
 * pn_verify_workspace_bytes of device memory (16-byte aligned), overwritten, with any content to
 * begin with; calls that may overlap need one each. */
#define PN_VERIFY_MAX_DRAFTS 63
int64_t pn_verify_workspace_bytes(int64_t B, int64_t V);

int pn_verify(int type, const void *p, int64_t p_stride, const void *q, int64_t q_stride,
              const int32_t *draft, const int32_t *n_draft, const float *u_accept,
              const float *u_sample, int64_t B, int64_t K, int64_t V, int32_t *tokens,
              int32_t *accepted, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PN_H */

/*
 * warp_decode_block.h -- C ABI of the operators around the MoE layer in a
 * decoder block: dense projections with 4-bit weights, a paged KV cache held
 * in 4 bits with the attentions that read it, rotary positions, and the norms
 * that join a block to the residual stream. Same library, statuses and conventions as
 * warp_decode.h: the caller owns every device buffer, nothing is allocated or
 * synchronised, work is enqueued on `stream`, what the host can see wrong
 * launches nothing, and moe_last_error() says why.
 *
 * 4-bit data is MXFP4 (OCP MX v1.0): E2M1 codes (sign, two exponent bits, one
 * mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), one E8M0 scale 2^(s-127) per 32
 * consecutive elements (s = 255 makes the block NaN). The quantisers here use
 * the conversion of OCP MX v1.0, as moe_pack_weights does for MXFP8: shared
 * exponent floor(log2(max|v|)) - 2, clamped to [-127, 127]; an all-zero block
 * stores s = 0; elements v / 2^exponent rounded to the nearest E2M1, ties to
 * even, magnitudes above 6 saturated. A block that holds an infinity or a NaN
 * stores s = 255. Every step is exact but the one rounding, so the codes do
 * not depend on the device.
 *
 * Strides ("ld...") are in elements; the last axis of every tensor is dense.
 */
#ifndef WARP_DECODE_BLOCK_H
#define WARP_DECODE_BLOCK_H

#include "warp_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { WD_F32 = 0, WD_BF16 = 1, WD_F16 = 2 } wd_dtype;

/* ------------------------------------------------ 4-bit projections -- */

/* W [N][K]: N >= 1 output rows, K % 32 == 0, 32 <= K <= 65536. */
typedef struct {
  int32_t N, K;
} wd_fp4_shape;

/* Packed weights, device memory, written by the two packers below. With
 * row tiles of 16 (N padded with zero rows) and column tiles of 128 (K padded
 * with zero codes and scales):
 *   codes  [N/16][K/128][16 rows][4 t][4 blocks][4 bytes]: byte j of (t, b) holds
 *          elements 32b + 8t + 2j (low nibble) and 32b + 8t + 2j + 1 (high) of
 *          the column tile;
 *   scales [N/16][K/128][8 g][2 h][4 blocks]: of row g + 8h of the tile.
 * Both 32-byte aligned. */
enum { WD_FP4_CODES = 0, WD_FP4_SCALES = 1 };

/* Bytes of packed array `which`; 0 if the shape is invalid or `which` unknown. */
size_t wd_fp4_packed_bytes(const wd_fp4_shape* shape, int which);

/* Pack an MXFP4 checkpoint: codes [N][K/2] (even element in the low nibble)
 * and scales [N][K/32], row-major, into the layout above. */
moe_status wd_fp4_pack_codes(const wd_fp4_shape* shape, const uint8_t* codes,
                             const uint8_t* scales, uint8_t* packed_codes,
                             uint8_t* packed_scales, void* stream);

/* Quantise w [N][K] (w_type, row stride ldw) to MXFP4 and pack it. */
moe_status wd_fp4_pack_weights(const wd_fp4_shape* shape, const void* w, int32_t w_type,
                               int64_t ldw, uint8_t* packed_codes, uint8_t* packed_scales,
                               void* stream);

/*
 * wd_fp4_matvec -- y[b,n] = sum_k x[b,k] W[n,k] for the B tokens of a decode
 * batch. x [B][K] BF16 or F16, 16-byte aligned with ldx % 8 == 0; y [B][N] F32,
 * BF16 or F16. Products are exact, sums FP32, y is rounded once. F16 values of x are
 * used exactly, BF16 ones down to 2^-31 of their token's largest finite one; below that
 * they are off by at most 2^-39 of it. Any scales may stand beside one another in a row (with more
 * than 8 tokens, blocks below 2^-26 of their row's largest scale are slower, where
 * they are not zeros; so are calls with results that are not finite). Up to 8
 * tokens one kernel streams the weights through mma.sync; more go through tcgen05,
 * 64 at a time, 32 above K = 8192, 16 above K = 16384, or 8 at a time through the
 * first above K = 32768. The results are the same on every call; a token's do not
 * depend on the other tokens' values, but their order of summation does on the
 * batch's size.
 */
moe_status wd_fp4_matvec(const wd_fp4_shape* shape, const uint8_t* packed_codes,
                         const uint8_t* packed_scales, const void* x, int32_t x_type,
                         int64_t ldx, int32_t B, void* y, int32_t y_type, int64_t ldy,
                         void* stream);

/* ------------------------------------------------------ 4-bit KV cache -- */

/* One layer's paged cache: `pages` pages of page_size tokens (16, 32, 64, 128
 * or 256), `heads` KV heads of `dim` elements (64, 128 or 256), quantised along
 * dim. Per (page, head), with key = slot in the page, pair = key / 2:
 *   k_codes  [page_size][4 t][dim/32 blocks][4 bytes]: byte j of (t, b) holds
 *            elements 32b + 8t + 2j (low nibble), + 1 (high)
 *   k_scales [page_size][dim/32]
 *   v_codes  [page_size/2 pairs][8 g][dim/32 blocks][4 bytes]: byte j of (g, b)
 *            holds element 32b + 4g + j of key 2 pair (low nibble), 2 pair + 1 (high)
 *   v_scales [page_size/2 pairs][dim/32][2 keys]
 * Arrays [pages][heads][...], each 16-byte aligned. */
typedef struct {
  int32_t pages, page_size, heads, dim;
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
} wd_kv4_cache;

enum { WD_KV4_CODES = 0, WD_KV4_SCALES = 1 };

/* Bytes of the codes or of the scales of K (and the same for V); 0 if the
 * cache's four sizes are invalid. The pointers are not looked at. */
size_t wd_kv4_cache_bytes(const wd_kv4_cache* cache, int which);

/*
 * The S sequences of a call: block_table [S][max_blocks] int32, entry j of a
 * row the page that holds its positions j*page_size ...; seq_lens [S] int32.
 * A page outside [0, pages), a negative length and a position beyond
 * max_blocks * page_size are not touched: they set bit 0 of *err_flag, if
 * err_flag is non-NULL, and what they would hold is left out.
 *
 * wd_kv4_append -- quantise the T new tokens' k and v [T][heads][dim] (type,
 * token strides ldk and ldv, multiples of 8, 16-byte aligned) into the cache.
 * Sequence s holds seq_lens[s] tokens before the call; its new ones are rows
 * cu_new[s] ... cu_new[s+1]-1 of k and v (cu_new [S+1] int32, not decreasing).
 * Rows from cu_new[S] on are ignored. cu_new NULL: one new token each (T == S).
 * Two sequences must not append to the same slot; neighbouring slots of a page
 * are independent, although their V shares bytes. T and S are below 2^31 - 2^16.
 *
 * wd_kv4_gather -- the reverse with the same arguments: the values of positions
 * seq_lens[s] ... of each sequence as k_out and v_out. Every MXFP4 value is
 * exact in BF16 and F32 but NaN blocks; F16 rounds, and overflows to infinity.
 * Rows that are ignored or left out are not written.
 */
moe_status wd_kv4_append(const wd_kv4_cache* cache, const void* k, const void* v, int32_t type,
                         int64_t ldk, int64_t ldv, int32_t T, const int32_t* block_table,
                         int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_new,
                         int32_t S, int32_t* err_flag, void* stream);
moe_status wd_kv4_gather(const wd_kv4_cache* cache, void* k_out, void* v_out, int32_t type,
                         int64_t ldk, int64_t ldv, int32_t T, const int32_t* block_table,
                         int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_new,
                         int32_t S, int32_t* err_flag, void* stream);

/*
 * wd_kv4_attend -- attention of one query token per sequence over the cache:
 *   z_j = scale * q . k_j  for the keys j in [max(0, len - window), len)
 *   out = sum_j softmax(z)_j v_j,  lse = log sum_j exp(z_j)
 * with len = seq_lens[s] (the token itself included) and window 0 for all keys.
 * q [S][q_heads][dim] BF16 or F16 (token stride ldq, a multiple of 8, 16-byte
 * aligned), q_heads a multiple of the cache's heads: query head h reads KV head
 * h / (q_heads / heads). out [S][q_heads][dim] of q's type (token stride ldo, a
 * multiple of 8, 16-byte aligned); lse [S][q_heads] F32 or NULL. A sequence
 * without keys gets out = 0 and lse = -inf. Results are the same on every call
 * with the same inputs.
 * Logits, softmax statistics and sums are FP32; q is used as exactly as x above (per head). The weight of a value's block, its
 * probability times its E8M0 scale, has 16 bits and FP32's range of exponents: a
 * probability below 2^-126 of the row's largest counts as 0, and a weight below 2^-140
 * of the largest probability times the block's largest scale among the keys. Keys and
 * values of up to 2^100 in magnitude do not overflow a sum on the way.
 * workspace: wd_kv4_attend_workspace bytes, 16-byte aligned; its contents do not
 * matter before or after a call. Calls that may overlap need one each.
 * pages * heads * (page_size / 16) < 2^31, 1 TB of codes.
 */
size_t wd_kv4_attend_workspace(const wd_kv4_cache* cache, int32_t S, int32_t q_heads);
/* The CTAs that a call with these sizes launches, at most 2 per SM; 0 where it launches
 * none: nothing to do, or refused. The pointers are not looked at. */
int32_t wd_kv4_attend_ctas(const wd_kv4_cache* cache, int32_t S, int32_t q_heads,
                           int32_t max_blocks, int32_t window);
moe_status wd_kv4_attend(const wd_kv4_cache* cache, const void* q, int32_t type, int64_t ldq,
                         int32_t S, int32_t q_heads, const int32_t* block_table,
                         int32_t max_blocks, const int32_t* seq_lens, float scale,
                         int32_t window, void* out, int64_t ldo, float* lse, void* workspace,
                         size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * wd_kv4_attend_chunk -- attention of several new tokens per sequence over the
 * cache, which holds them already: prompts, chunks of prompts, drafts to verify.
 * T, block_table, seq_lens, cu_new and S are wd_kv4_append's: row cu_new[s] + i of q
 * is at position p = seq_lens[s] + i (seq_lens without the new tokens) and attends to
 *   z_j = scale * q . k_j  for the keys j in [max(0, p + 1 - window), p]
 *   out = sum_j softmax(z)_j v_j,  lse = log sum_j exp(z_j)
 * with window 0 for all keys up to p. q [T][q_heads][dim] BF16 or F16 (token stride
 * ldq, a multiple of 8, 16-byte aligned), q_heads a multiple of the cache's heads:
 * query head h reads KV head h / (q_heads / heads). out [T][q_heads][dim] of q's type
 * (token stride ldo, a multiple of 8, 16-byte aligned); lse [T][q_heads] F32 or NULL.
 * Rows of q that belong to no sequence (in front of cu_new[0], from cu_new[S] on) are
 * ignored: their out and lse are not written. A row that sees no key (a negative
 * length, none of its pages valid) gets out = 0 and lse = -inf. A key that a row does
 * not see has no influence on it, NaN and infinities included. Results are the same on
 * every call with the same inputs.
 * Logits, softmax statistics and sums are FP32; q is used as in wd_kv4_attend. Keys are used
 * exactly, but for a key with scale codes outside 109 .. 136: its blocks 2^-36 below its
 * largest are rounded to that, and lower ones count as 0. A probability has 16 bits, fewer
 * below 2^-118 of its row's largest; below 2^-126 of that it counts as 0. Keys and
 * values of up to 2^100 in magnitude do not overflow a sum on the way.
 * workspace: wd_kv4_attend_chunk_workspace bytes for T tokens or more, 16-byte aligned;
 * its contents do not matter before or after a call. Calls that may overlap need one
 * each. The kernel's waits for copies and products have a limit; were one to run out, results
 * would be NaN (err_flag only tells of lengths and pages). max_blocks * page_size < 2^31 - 2^16,
 * T * q_heads and S < 2^31 - 2^16, q_heads <= 65536.
 */
size_t wd_kv4_attend_chunk_workspace(const wd_kv4_cache* cache, int32_t T, int32_t q_heads);
moe_status wd_kv4_attend_chunk(const wd_kv4_cache* cache, const void* q, int32_t type,
                               int64_t ldq, int32_t T, int32_t q_heads,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seq_lens, const int32_t* cu_new, int32_t S,
                               float scale, int32_t window, void* out, int64_t ldo, float* lse,
                               void* workspace, size_t workspace_bytes, int32_t* err_flag,
                               void* stream);

/* ---------------------------------------------------- rotary positions -- */

/* How heads turn with their tokens' positions. rot_dim elements of a head (its
 * first; a multiple of 16) form rot_dim / 2 pairs: pair i is elements i and
 * i + rot_dim / 2, or, where neighbours is not 0, 2i and 2i + 1. At position p it
 * turns by the angle p * f_i and is multiplied by magnitude (0, or 2^-100 to 65536 in size):
 *   a' = magnitude (a cos - b sin),   b' = magnitude (b cos + a sin)
 * turns [rot_dim/2] (device memory, 8 bytes aligned): f_i as turns per position
 * times 2^64, modulo whole turns, written on the host by wd_rope_turns. */
typedef struct {
  int32_t rot_dim, neighbours;
  double magnitude;
  const uint64_t* turns;
} wd_rotation;

/* The n frequencies (radians per position, at most 65536 in magnitude) as a
 * rotation keeps them; both arrays in host memory. */
moe_status wd_rope_turns(int32_t n, const double* freqs, uint64_t* turns);

/*
 * wd_rope -- turn the heads of x [T][heads][dim] (F32, BF16 or F16; dim a
 * multiple of 8 up to 1024) by positions [T] int32 into out. Negative positions
 * turn back. Elements behind rot_dim are copied. out may be x (with the same
 * stride); token strides ldx and ldo a multiple of 16 bytes, as the addresses.
 * Angles are exact to 2^-23 whatever the position; with these and FP32 results are
 * off by 6 * 2^-24 (|a| + |b|) magnitude before their one rounding.
 */
moe_status wd_rope(const wd_rotation* rotation, const void* x, int32_t type, int64_t ldx,
                   int32_t T, int32_t heads, int32_t dim, const int32_t* positions, void* out,
                   int64_t ldo, void* stream);

/*
 * wd_kv4_rope_append -- wd_kv4_append with the rotation on its way: k turned by
 * its tokens' positions (seq_lens[s] + the token's number among the new ones) and
 * quantised, v quantised, q [T][q_heads][dim] turned into q_out (which may be q
 * with the same stride; type and strides as k's; q_heads 0: no queries).
 * The cache holds the nearest MXFP4 to the exact turned key, not to one rounded to
 * the input's type before (for blocks whose largest input is 2^-100 or more; FP32's
 * infinity, which a turn of the largest finite BF16 can reach, makes a block NaN).
 * What wd_kv4_append leaves out is left out here; a query without a place in the
 * cache is turned all the same, one that is ignored or whose sequence has a
 * negative length is not written.
 */
moe_status wd_kv4_rope_append(const wd_kv4_cache* cache, const wd_rotation* rotation,
                              const void* q, int64_t ldq, int32_t q_heads, void* q_out,
                              int64_t ldqo, const void* k, const void* v, int32_t type,
                              int64_t ldk, int64_t ldv, int32_t T, const int32_t* block_table,
                              int32_t max_blocks, const int32_t* seq_lens,
                              const int32_t* cu_new, int32_t S, int32_t* err_flag, void* stream);

/* --------------------------------------------------------- block norms -- */

/*
 * wd_block_norm -- the step between two blocks of a decoder layer, for T tokens
 * of H channels (1 <= H <= 8192):
 *   r' = res_scale * res + gate * N(y; w_post)      N(v; w) = v w / sqrt(mean(v^2) + eps)
 *   out = N(r'; w_pre)                              (from r' before its rounding)
 * y is the output of the block before, out the input of the one behind, res
 * the residual stream. Any of the parts may be missing (NULL): y (r' =
 * res_scale * res), w_post (y itself is added), gate (1), w_pre (then out must
 * be NULL, and the other way round), res_out (r' is not kept). gate is
 * read at token * gate_ld + channel * gate_step: 0 broadcasts along an axis.
 * Types: res and res_out res_type; y y_type; w_post [H], w_pre [H] and gate
 * w_type; out out_type (each F32, BF16 or F16). Everything is computed in FP32
 * and rounded once. res_out may be res; out may be y or res where the types,
 * strides and addresses are the same.
 */
moe_status wd_block_norm(int32_t T, int32_t H, const void* res, int32_t res_type, int64_t ldr,
                         const void* y, int32_t y_type, int64_t ldy, const void* w_post,
                         const void* w_pre, const void* gate, int32_t w_type, int64_t gate_ld,
                         int32_t gate_step, float res_scale, float eps, void* res_out,
                         int64_t ldro, void* out, int32_t out_type, int64_t ldo, void* stream);

/* ------------------------------------------------- arguments as a block -- */

/* wd_call -- the entry point `which` with its arguments, 8 bytes each, in their
 * order: integers and pointers as int64, floats as double. For bindings that pay
 * per argument; the result and the errors are the entry point's. An int32 argument
 * whose word holds more is refused (MOE_ERR_SHAPE). */
enum {
  WD_CALL_FP4_MATVEC = 0,
  WD_CALL_KV4_APPEND = 1,
  WD_CALL_KV4_GATHER = 2,
  WD_CALL_KV4_ATTEND = 3,
  WD_CALL_BLOCK_NORM = 4,
  WD_CALL_ROPE = 8, /* a number once given stays its entry point's; 5 to 7 never were one */
  WD_CALL_KV4_ROPE_APPEND = 9,
  WD_CALL_KV4_ATTEND_CHUNK = 10
};
moe_status wd_call(int32_t which, const void* args);

#ifdef __cplusplus
}
#endif

#endif /* WARP_DECODE_BLOCK_H */

/*
 * mla_kv_q8.h — C ABI of the 8-bit latent cache: appending rows with the position rotation,
 * tree-verify attention over e4m3 rows, and their defragmenting gather.
 *
 * The cache.  kv_cache is e4m3 [num_slots][576] (one byte a value: 512 latent dims, then 64
 * rope dims), page size 1.  Slots [i * scale_block, (i + 1) * scale_block) share the fp32
 * scale scales[i]; scale_block is a power of two from 1 (a scale for every row, the form that
 * mla_kv_append() computes) up to 2^30 (one scale for the whole cache).  A stored code x
 * stands for x * scales[slot / scale_block].  A valid scale lies in [2^-40, 2^40].
 *
 * Return codes, ownership and capture rules are those of mla_tree_verify.h: every buffer is
 * the caller's, nothing is allocated, synchronised or read back, every call only enqueues
 * kernels on the given stream and can be captured in a CUDA graph.
 */
#ifndef MLA_KV_Q8_H_
#define MLA_KV_Q8_H_

#include "mla_tree_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_KV_TYPE_BF16 0
#define MLA_KV_TYPE_E4M3 1

/* Further device error bit of mla_tree_verify_q8(), beside MLA_TV_DEV_*. */
#define MLA_TV_DEV_BAD_SCALE 16u  /* the scale of a referenced slot is NaN or outside
                                     [2^-40, 2^40]: that key is skipped, as if masked */

/*
 * mla_kv_append — writes the cache rows of n new tokens, rotating their rope dims by the
 * token's position, and optionally rotates the rope part of the tokens' queries.
 *
 * Token i with slot s = slots[i] and position p = positions[i]:
 *   (c_k, s_k) = (cos_sin[p][k], cos_sin[p][32 + k]),  k = 0..31
 *   pair k of a 64-vector x is (x[2k], x[2k+1]) when `interleaved`, else (x[k], x[k+32]);
 *   rot(x) maps pair (a, b) to (a c_k - b s_k, b c_k + a s_k), computed in fp32
 *   row = [latent[i][0:512], rot(k_pe[i][0:64])]
 *   bf16 cache:  kv_cache[s] = row, rounded to nearest even
 *   e4m3 cache:  kv_cache[s] = e4m3(row * (1 / scale)), rounded to nearest even, saturated
 *     to +-448, where scale is, with given_scales = 0 (needs scale_block = 1),
 *       scales[s] = max(max|row| / 448, 2^-40), or 1 for a row of zeros (written);
 *     with given_scales = 1, scales[s / scale_block] as it stands (read only).
 *   q_out[i][h] = bf16(rot(q_pe[i][h])) for every head h, when q_pe is not NULL
 * A token with slot -1 is padding: nothing is written for it, its q_out included.
 * Two tokens with the same slot leave that slot's row and scale undefined (other rows are
 * not affected); rows and scales that no token names are left as they were.
 *
 *   latent       bf16, rows latent_stride elements apart; 16-byte aligned, stride a multiple
 *                of 8
 *   k_pe         bf16, rows k_pe_stride elements apart, 2-byte aligned (latent and k_pe may be
 *                slices of one projection's output)
 *   positions    int64 [n]
 *   cos_sin      fp32 [max_pos][64]: 32 cosines, then 32 sines
 *   slots        int64 [n]
 *   kv_cache     cache_type MLA_KV_TYPE_BF16: bf16 [num_slots][576]; _E4M3: as above;
 *                contiguous, 16-byte aligned
 *   scales       fp32 [ceil(num_slots / scale_block)]; must be NULL for a bf16 cache
 *   q_pe, q_out  bf16 [n][num_heads][64] with element strides between tokens and heads
 *                (both NULL: no queries); 16-byte aligned, strides multiples of 8.  q_out may
 *                be the last 64 dims of the q of mla_tree_verify(); the two must not overlap
 *                except by being the same view
 *   status       device uint32 the caller zeroes once; the kernel ORs in
 *                MLA_KV_APPEND_BAD_SLOT (a slot below -1 or past num_slots) and _BAD_POS (a
 *                position outside [0, max_pos)): such a token is skipped like padding;
 *                _BAD_VALUE: a row holds a NaN or an infinity, or computed scales would pass
 *                2^40 (with computed scales the row is written as NaN codes with scale 1, so
 *                that attention that sees it gives NaN; with given scales the values that are
 *                NaN or infinite become NaN codes; a bf16 row is written as it is);
 *                _BAD_SCALE: a given scale is NaN or
 *                outside [2^-40, 2^40] (the token is skipped like padding)
 *
 * Returns MLA_TV_OK (n = 0 enqueues nothing), or before enqueuing anything MLA_TV_ERR_NULL /
 * _SHAPE (n < 0, num_slots outside [1, INT32_MAX], max_pos < 1, an unknown cache_type, a
 * scale_block that is no power of two in [1, 2^30], given_scales = 0 with scale_block > 1,
 * num_heads outside [1, 1024] with queries, a negative stride, or more than 2^31 warps of
 * work) / _ALIGN / _DEVICE, or MLA_TV_ERR_LAUNCH.
 */
#define MLA_KV_APPEND_BAD_SLOT 1u
#define MLA_KV_APPEND_BAD_POS 2u
#define MLA_KV_APPEND_BAD_VALUE 4u
#define MLA_KV_APPEND_BAD_SCALE 8u
int mla_kv_append(const void* latent, int64_t latent_stride, const void* k_pe, int64_t k_pe_stride,
                  const int64_t* positions, const float* cos_sin, int64_t max_pos,
                  const int64_t* slots, void* kv_cache, int32_t cache_type, float* scales,
                  int64_t scale_block, int32_t given_scales, int64_t num_slots, const void* q_pe,
                  int64_t q_pe_token_stride, int64_t q_pe_head_stride, void* q_out,
                  int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t num_heads,
                  int64_t n, int32_t interleaved, uint32_t* status, cudaStream_t stream);

/* Bytes of workspace of mla_tree_verify_q8(): that of mla_tree_verify() and room for the
 * split queries (bs * max_q_per_req * num_heads rows of 1156 bytes, fewer than 2^30).  0 for
 * arguments that the call refuses. */
size_t mla_tree_verify_q8_workspace_bytes(int32_t bs, int32_t max_q_per_req, int32_t num_heads);

/*
 * mla_tree_verify_q8 — mla_tree_verify() over the e4m3 cache: the same batch description,
 * visibility, outputs and error handling, with
 *   kv_cache     e4m3 [num_slots][576], contiguous, 16-byte aligned
 *   scales       fp32 [ceil(num_slots / scale_block)]
 *   scale_block  slots that share a scale
 * A request with one token (T_b = 1) is plain decoding.  For key column c with scale g(c),
 *   s_c = sm_scale * g(c) * <q[r,h,0:576], code(c)[0:576]>
 *   out[r,h,0:512] = softmax over visible c of s_c, applied to g(c) * code(c)[0:512]
 * A NaN code in a row that a query token does not see does not reach that token's output;
 * one in a row that it sees makes its output and lse NaN.
 * Precision, beside fp32 sums and out's bf16: a query row's values are exact down to 2^-9 of its
 * largest and within 2^-17 of that below; a key's weight w_c is off by at most 2^-8 + 2^-11 of
 * itself, as in bf16, while w_c g(c) is at least 2^-13 of the largest w g of the column's keys
 * that hold any latent value, and smaller ones are rounded at random to the right mean (off by at
 * most a quarter, and from 2^-21 on down by a step of 2^-23 of that largest).  lse does not depend
 * on those roundings.  The same call gives the same bits.
 * Reads the device error bits with
 * mla_tree_verify_read_device_status(); MLA_TV_DEV_BAD_SCALE may be among them.
 */
int mla_tree_verify_q8(const void* q, const void* kv_cache, const float* scales,
                       const int32_t* kv_indices, const int32_t* kv_indptr,
                       const int64_t* out_cache_loc, const uint8_t* custom_mask,
                       const int64_t* mask_indptr, const int64_t* qo_indptr, float sm_scale,
                       void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t bs,
                       int32_t max_q_per_req, int32_t num_heads, int64_t num_slots,
                       int64_t total_q, int64_t num_kv_indices, int64_t mask_len,
                       int64_t scale_block, cudaStream_t stream);

/*
 * The same with the debug settings of mla_tree_verify_debug_ex() that this kernel has:
 * wait_limit_ns and lanes.  The dumps must be NULL and merge_mode MLA_TV_MERGE_AUTO, else
 * MLA_TV_ERR_SHAPE; opts must not be NULL.
 */
int mla_tree_verify_q8_debug_ex(const void* q, const void* kv_cache, const float* scales,
                                const int32_t* kv_indices, const int32_t* kv_indptr,
                                const int64_t* out_cache_loc, const uint8_t* custom_mask,
                                const int64_t* mask_indptr, const int64_t* qo_indptr,
                                float sm_scale, void* out, float* lse, void* workspace,
                                size_t workspace_bytes, int32_t bs, int32_t max_q_per_req,
                                int32_t num_heads, int64_t num_slots, int64_t total_q,
                                int64_t num_kv_indices, int64_t mask_len, int64_t scale_block,
                                const mla_tree_verify_debug_opts* opts, cudaStream_t stream);

/*
 * mla_tree_verify_q8() with settings for the merge of the pieces that a query token's keys are
 * cut into (test hooks; the output bits are the same with all of them):
 *   merge_mode     MLA_TV_Q8_MERGE_AUTO: as timing allows (the normal call: the CTA of the last
 *                  piece merges from TMEM if the others are done before it, else CTAs without
 *                  work left share the merge).  _NO_TMEM: never from TMEM.  _ALONE: the CTA that
 *                  finishes last merges, from the workspace and alone.
 *   help_limit_ns  how long a CTA without work left waits for the other pieces before it leaves
 *                  the merge to others: 0 the library's choice (40 us), at most 10^9
 * Others give MLA_TV_ERR_SHAPE.
 */
#define MLA_TV_Q8_MERGE_AUTO 0
#define MLA_TV_Q8_MERGE_NO_TMEM 1
#define MLA_TV_Q8_MERGE_ALONE 2
int mla_tree_verify_q8_debug_merge(const void* q, const void* kv_cache, const float* scales,
                                   const int32_t* kv_indices, const int32_t* kv_indptr,
                                   const int64_t* out_cache_loc, const uint8_t* custom_mask,
                                   const int64_t* mask_indptr, const int64_t* qo_indptr,
                                   float sm_scale, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, int32_t bs, int32_t max_q_per_req,
                                   int32_t num_heads, int64_t num_slots, int64_t total_q,
                                   int64_t num_kv_indices, int64_t mask_len, int64_t scale_block,
                                   int32_t merge_mode, int64_t help_limit_ns, cudaStream_t stream);

/*
 * mla_kv_gather_q8 — mla_tree_verify_kv_gather() for an e4m3 cache with a scale for every
 * row (scale_block = 1): for every index entry i in [kv_indptr[0], kv_indptr[bs]), with
 * j = i - kv_indptr[0],
 *   dst row j = kv_cache row kv_indices[i] (576 bytes, bit for bit), dst_scales[j] =
 *   scales[kv_indices[i]], new_indices[i] = dst_slot0 + j
 * A slot outside [0, num_slots) gives a row of zeros with scale 1, flagged.  Arguments,
 * status bits (MLA_TV_GATHER_*), overlap rule and return codes are those of
 * mla_tree_verify_kv_gather(); scales and dst_scales are fp32 [num_slots] and [dst_rows].
 */
int mla_kv_gather_q8(const void* kv_cache, const float* scales, int64_t num_slots,
                     const int32_t* kv_indices, int64_t num_kv_indices, const int32_t* kv_indptr,
                     int32_t bs, void* dst, float* dst_scales, int64_t dst_rows,
                     int32_t dst_slot0, int32_t* new_indices, uint32_t* status,
                     cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_KV_Q8_H_ */

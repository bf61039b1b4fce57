/*
 * exact_attention_51_gb300 -- C ABI of the paged e4m3 key/value cache:
 * appending to it and attending over it.
 *
 * The cache is a pool of pages of `page_size` tokens:
 *
 *     k_cache, v_cache  e4m3 codes [num_pages, Hkv, page_size, d]
 *     k_scale, v_scale  fp32 [num_pages, Hkv]
 *
 * Element x of a page and head means scale * x.  Scales are powers of two from
 * 2^-60 to 2^60, the ones that attn_paged_append_fp8 writes: a block whose
 * scale has to grow then keeps its codes exactly (but for those that leave the
 * type's normal range), however often it grows.  attn_fwd_fp8_paged reads
 * scales of any other value in that range too.  Of a sequence and head it wants
 * V's scales within 2^100 of each other: a key whose weight times V scale is
 * less than 2^-133 of the largest such product is left out, which within that
 * spread is no weight above 2^-33 of the largest.
 *
 * A sequence's tokens lie in the pages that its row of the page table names:
 * token j is token j % page_size of page block_table[b][j / page_size].
 * Sequences may share pages for reading.
 *
 * Device-side indexes (slots, page numbers, sequence starts) cannot be checked
 * on the host.  The kernels check them: what lies outside of its buffer is
 * neither read nor written, and a code in the device status word says so
 * (attn_fwd_device_status, ATTN_ERR_BAD_INDEX).
 *
 * Conventions (status codes, streams, ownership, thread safety) as in
 * include/attn_fwd.h.
 */
#ifndef EXACT_ATTENTION_51_GB300_ATTN_PAGED_H
#define EXACT_ATTENTION_51_GB300_ATTN_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Appends T tokens' keys (rotated on the way) and values to the cache.
 *
 *   k, v       bf16 [T, Hkv, d], elements of a head adjacent, tokens and heads
 *              at the given strides (elements, multiples of 8, >= 0); 16-byte
 *              aligned.  d = 64, 128 or 256.
 *   slots      device int32 [T]: token t goes to token slots[t] % page_size of
 *              page slots[t] / page_size; a negative slot skips the token
 *              (padding).  Tokens of one page must be adjacent in t, in the order of
 *              their slots and without gaps, and no page may get tokens twice in a call
 *              (a sequence's new tokens in order satisfy this; a page for which it does not
 *              hold gets unspecified contents, other pages do not change by it).
 *   positions  device int32 [T]: the positions that keys are rotated by.
 *   phases, rot_dim, interleaved, attention_factor: the rotation, as in
 *              attn_rope; phases NULL (positions may then be NULL): keys are stored as
 *              they are.
 *   page_size  16, 32, 64 or 128.
 *   k_cache, v_cache  16-byte aligned; scales 4-byte aligned.
 *
 * Each block (page and head) that gets tokens takes the smallest scale of two's
 * powers whose 448 multiples hold its largest finite new value, but no smaller than the
 * scale that it had, where its earlier tokens stay: those before the first new
 * slot do, and their codes are rewritten for a larger scale (rounded to the
 * nearest).  A block written from its token 0 on starts anew.  Codes behind the
 * new tokens are left as they are.  The rotation is fp32 and each value is
 * rounded once, to the nearest e4m3 (ties to even; beyond 448 * 2^60: clamped).
 * Infinities and NaN are stored as NaN and leave the scale alone.
 *
 * k_cache, v_cache and the scales must not overlap each other or the inputs
 * (ATTN_ERR_ALIAS).  A slot beyond num_pages * page_size is skipped and
 * sets 0x201 in the status word.  T = 0 does nothing.  Enqueues one kernel.
 */
ATTN_API int attn_paged_append_fp8(const void* k, const void* v, int T, int Hkv, int d,
                                   int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
                                   int64_t v_stride_h, const int32_t* slots,
                                   const int32_t* positions, const uint64_t* phases, int rot_dim,
                                   int interleaved, float attention_factor, void* k_cache,
                                   void* v_cache, float* k_scale, float* v_scale, int num_pages,
                                   int page_size, void* stream);

/*
 * Attention of a ragged batch's newest tokens over the cache, with shared key
 * heads: query head h reads key head h / (Hq / Hkv).
 *
 *   q          bf16 [T, Hq, d], tokens and heads at the given strides
 *              (elements, multiples of 8, >= 0); 16-byte aligned.  d = 64, 128, 256.
 *   q_start    device int32 [B + 1], ascending from >= 0 to <= T: the query
 *              tokens of sequence b are q_start[b] .. q_start[b+1].  NULL: T / B
 *              tokens each (T a multiple of B).
 *   kv_len     device int32 [B]: keys of each sequence, its queries' own among them.
 *              0 is allowed (less counts as 0).
 *   block_table  device int32 [B, table_stride]: page numbers; entries from
 *              ceil(kv_len / page_size) on are not used.
 *   max_q      no sequence has more query tokens (1 for decoding; a larger one
 *              than need be costs time, as it picks the kernel and its tiles).
 *   max_kv     about the longest kv_len: only the sharing out of the keys goes by it,
 *              and the result does not depend on it.
 *   causal     query i of n sees keys j <= i + kv_len - n (the queries are the
 *              sequence's last n positions, as attn_fwd_kvcache); otherwise all kv_len.
 *   o          bf16 [T, Hq, d] contiguous, 16-byte aligned.  lse: fp32 [T, Hq].
 *              A query that sees no key gets O = 0 and LSE = -inf.  Rows of tokens
 *              outside of q_start[0] .. q_start[B] are left as they were.
 *   num_splits 1..64: shares of the keys that thread blocks of their own take
 *              (attn_fwd_fp8_paged_num_splits suggests a count).  With 1, a last wave
 *              of few blocks of many rows may still share out its keys.
 *   workspace  attn_fwd_fp8_paged_workspace_size(T, Hq, Hkv, d, max_q, num_splits) bytes,
 *              256-byte aligned; NULL where that is 0.  Scratch until the call's last
 *              kernel has run: calls that may overlap need one each.
 *
 * Scores are fp32 sums of exact products of the codes and Q, whose elements are
 * held to 2^-25 (up to 16 rows) or 2^-21 (more) of their row's largest, exactly
 * from 2^-13 of it on; a weight is rounded to fp16 (2^-11 of itself) where it
 * meets V, and O once to bf16.
 *
 * Masked keys do not reach the result, whatever their codes (NaN among them)
 * and scales.  Codes of tokens from kv_len on are never used.
 * Page numbers outside of [0, num_pages) and lengths beyond the table hide their tokens and set
 * 0x202 in the status word; sequence starts out of order or beyond T hide the
 * sequence, and more than max_q query tokens are left out, with 0x203.
 * Enqueues one kernel, and a merge where there is a workspace.  Up to 16 rows
 * (max_q * Hq / Hkv) of a sequence and key head run a kernel that reads the keys
 * once for all of them (its grid takes at most 65535 sequences and 65535 key
 * heads), more run on the tcgen05 tensor cores.
 */
ATTN_API int attn_fwd_fp8_paged(const void* q, int64_t q_stride_t, int64_t q_stride_h,
                                const void* k_cache, const void* v_cache, const float* k_scale,
                                const float* v_scale, const int32_t* block_table,
                                int table_stride, const int32_t* q_start, const int32_t* kv_len,
                                void* o, float* lse, int B, int T, int Hq, int Hkv, int d,
                                int num_pages, int page_size, int max_q, int max_kv, float scale,
                                int causal, int num_splits, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Workspace bytes: 0 for num_splits == 1, for up to 8 splits of at most 16
 * rows and up to 4 of more (a thread-block cluster merges those) and for invalid sizes, else num_splits *
 * T * Hq * (d + 1) * 4 bytes, each part 256-byte padded.  Host-only. */
ATTN_API size_t attn_fwd_fp8_paged_workspace_size(int T, int Hq, int Hkv, int d, int max_q,
                                                  int num_splits);

/* A split count for attn_fwd_fp8_paged on a GPU with `num_sms`
 * multiprocessors (1 for invalid sizes).  Host-only. */
ATTN_API int attn_fwd_fp8_paged_num_splits(int B, int Hq, int Hkv, int d, int page_size, int max_q,
                                           int max_kv, int num_sms);

/*
 * Self-test of the kernels' own abort path (a test hook, not a way to compute
 * attention), as attn_selftest_fwd_dropped_load: attn_fwd_fp8_paged on the given
 * arguments, except that one load never arrives in any thread block and every wait gives
 * up after `timeout_ms` (1..10000) milliseconds.  drop_load >= 0: up to 16 rows,
 * the ring's stage of that number (128 keys each, 64 at d = 256); more rows, 2 j
 * for the keys and 2 j + 1 for the values of the block's key tile j (128 keys, 64
 * at d = 256).  Blocks with fewer run to the end.  O and LSE are not valid
 * afterwards; attn_fwd_device_status returns ATTN_ERR_TIMEOUT with the code of the
 * wait that gave up first (0x14x up to 16 rows, 0x15x more) and clears the word.
 * Run it only when no other launch of the library is in flight on the device.
 */
ATTN_API int attn_selftest_fwd_fp8_paged_dropped_load(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache, const void* v_cache,
    const float* k_scale, const float* v_scale, const int32_t* block_table, int table_stride,
    const int32_t* q_start, const int32_t* kv_len, void* o, float* lse, int B, int T, int Hq, int Hkv,
    int d, int num_pages, int page_size, int max_q, int max_kv, float scale, int causal, int num_splits,
    void* workspace, size_t workspace_bytes, int drop_load, unsigned int timeout_ms, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_51_GB300_ATTN_PAGED_H */

// Host <-> kernel interface of attention over the paged e4m3 cache.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ea51 {

struct PagedParams {
  const __nv_bfloat16* q;
  long long qs_t, qs_h;  // strides in elements
  const uint8_t* k_cache;  // codes [num_pages, Hkv, page_size, D]
  const uint8_t* v_cache;
  const float* k_scale;    // [num_pages, Hkv]
  const float* v_scale;
  const int32_t* table;  // [B, table_stride]
  const int32_t* q_start;  // [B + 1], or nullptr: T / B tokens each
  const int32_t* kv_len;   // [B]
  __nv_bfloat16* o;  // [T, Hq, D]
  float* lse;        // [T, Hq]
  float* o_part;     // split-KV: [splits][T * Hq][D], normalised
  float* lse_part;   // [splits][T * Hq], natural log
  unsigned* status;  // [0] wait time-outs, [1] bad indexes
  int B, T, Hq, Hkv, group;
  int per_seq;    // query tokens a sequence without q_start
  int group_inv;  // ceil(2^16 / group)
  int table_stride, num_pages, page_size, page_shift;
  int max_q, tiles;  // row tiles of one sequence and key head (one, for the split-KV kernel)
  int splits, chunk;  // keys a split takes (the last one takes all that is left)
  int cluster;        // splits that a thread-block cluster merges in shared memory
  int shares;         // splits / cluster: partial results that the merge kernel joins
  int tail_tile;      // tcgen05 kernel: row tiles from here on, the last wave's, are a cluster's of two; 0: none
  int causal;
  float scale_log2;  // scale * log2(e)
  unsigned long long wait_timeout_ns;  // limit of each bounded wait
  int drop_load;  // a test hook: this load is left out (-1: none); see attn_selftest_fwd_fp8_paged_dropped_load
};

constexpr unsigned kCodeBadPage = 0x202, kCodeBadSequence = 0x203;

// Keys of the units that splits are cut in.
constexpr int kPagedUnit = 128;

// Largest cluster: splits up to it need no workspace and no merge kernel.
constexpr int kPagedCluster = 8;

// Rows of a tile from which on it is the tcgen05 kernel's (paged_prefill.cuh): a
// block of two tiles of 128 rows, one at d = 256.
constexpr int kPrefillRows = 128;

// Thread blocks on a multiprocessor.  Measured at d = 128 with 64-token pages, two and three: one
// sequence of 131072 keys 48 us and 52, 16 queries a block 226 and 294; with 16-token pages, 64
// sequences of up to 16384 keys 148 us and 131.
constexpr int paged_blocks(int d, int tile_rows, int page_size) {
  return tile_rows >= kPrefillRows ? 1 : page_size == 16 && (d <= 128 || tile_rows <= 8) ? 3 : 2;
}

// The same of the tcgen05 kernel, whose blocks fill a multiprocessor each: larger clusters do not
// fill a group of multiprocessors.
constexpr int kPrefillCluster = 4;

// First of the row tiles of the tcgen05 kernel that are left for a last, partial wave where blocks
// take whole tiles (0: all tiles alike).  Two blocks of a cluster share such a tile's keys: 2 x
// 2048 queries against 16384 keys are 512 tiles, three waves of 152 and 56 that two blocks each
// take (833 us, 911 without; 192 tiles at d = 64 293 and 367).  The launch is one of clusters of
// two, and those before take two tiles each: 152 multiprocessors hold 76 of them.  (Of four they
// would leave some empty in every wave.)  Where the tiles' keys differ much, as in a whole prompt,
// the longest come first and the short ones fill the gaps already (4096 against 4096, 32/8 heads of
// 128: 144 us, 149 with pairs).
inline long long paged_tail(long long tiles, int num_sms, long long max_q, long long max_kv, bool causal) {
  const long long first = tiles / num_sms * num_sms / 2 * 2, rest = tiles - first;
  // (below 2048 keys a share's begin, end and merge cost what it saves)
  if (first == 0 || rest == 0 || 2 * rest > num_sms || max_kv < 2048) return 0;
  return causal && 4 * max_q > max_kv ? 0 : first;
}

// Splits that a cluster takes: all or one.
inline int paged_cluster(int tile_rows, int splits) {
  return splits <= (tile_rows < kPrefillRows ? kPagedCluster : kPrefillCluster) ? splits : 1;
}

// Query rows (token, head of the group) of a block for sequences of `rows` rows:
// 8 or 16 of the split-KV kernel, 256 (d = 256: 128) of the tcgen05 kernel.  Measured,
// tiles of 32 rows of the former (16 sequences of 8192 keys, 32/8 heads of 128, 8 queries: 115 us; one of
// 32768: 40) are no faster than the latter's (107 and 39 us).
int paged_rows(int d, long long rows);

cudaError_t launch_paged(int d, int tile_rows, const CUtensorMap* tk, const CUtensorMap* tv,
                         const PagedParams& p, cudaStream_t stream);
cudaError_t launch_paged_combine(int d, const PagedParams& p, cudaStream_t stream);

// Rows of the TMA boxes: a page or a stage's keys.
int paged_box_rows(int d, int page_size);

}  // namespace ea51

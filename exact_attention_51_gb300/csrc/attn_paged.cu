// Attention over the paged e4m3 cache: the entry points of
// include/attn_paged.h, their checks, and the merge of split keys.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_paged.h"
#include "fwd_dispatch.h"
#include "paged_kernel.cuh"

namespace ea51 {

cudaError_t launch_paged_d64(int, const CUtensorMap*, const CUtensorMap*, const PagedParams&, cudaStream_t);
cudaError_t launch_paged_d128(int, const CUtensorMap*, const CUtensorMap*, const PagedParams&, cudaStream_t);
cudaError_t launch_paged_d256(int, const CUtensorMap*, const CUtensorMap*, const PagedParams&, cudaStream_t);

cudaError_t launch_paged(int d, int tile_rows, const CUtensorMap* tk, const CUtensorMap* tv,
                         const PagedParams& p, cudaStream_t stream) {
  return d == 64    ? launch_paged_d64(tile_rows, tk, tv, p, stream)
         : d == 128 ? launch_paged_d128(tile_rows, tk, tv, p, stream)
                    : launch_paged_d256(tile_rows, tk, tv, p, stream);
}

int paged_rows(int d, long long rows) {
  if (rows <= 8) return 8;
  if (rows <= 16) return 16;
  return d == 256 ? 128 : 256;
}

int paged_box_rows(int d, int page_size) { return std::min(page_size, d == 256 ? 64 : 128); }

namespace {

// O = sum_s exp(L_s - L) O_s over the shares that saw a key, as attn_combine_kernel.
// WARPS warps take a row, 8 / WARPS rows a block.  A decoding step has few rows
// and many shares: eight warps share out a row's (one warp reading 48 shares of 32 rows one after
// another took longer than the attention itself).  A prompt's chunk has many rows
// of a few shares: a warp each (4096 queries over 4096 keys in 2 shares, 32/8 heads of 128:
// 236 us with the attention, 462 with a block per row).
template <int D, int WARPS>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p) {
  constexpr int PER = D / 32, ROWS = 8 / WARPS;
  constexpr int WIDE = PER < 4 ? PER : 4;  // elements a load
  __shared__ float s_acc[WARPS > 1 ? WARPS : 1][WARPS > 1 ? D : 1];
  __shared__ float s_sum[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = warp % WARPS;
  chain_begin();
  const unsigned cell = blockIdx.x * ROWS + warp / WARPS;  // (key head, query row of its group) of a sequence
  const unsigned per_head = static_cast<unsigned>(p.max_q) * static_cast<unsigned>(p.group);
  const unsigned bh = cell / per_head, r = cell - bh * per_head;
  const int b = static_cast<int>(bh / static_cast<unsigned>(p.Hkv)), h = static_cast<int>(bh) - b * p.Hkv;
  if (b >= p.B) return;  // (with WARPS == 8 no block has such a row, so that all of a block's warps leave or none)
  const PagedSeq seq = paged_seq(p, b, false);
  if (static_cast<int>(r) >= min(seq.nq, p.max_q) * p.group) return;
  const int token = static_cast<int>(r) / p.group;
  const long long row =
      static_cast<long long>(seq.q0 + token) * p.Hq + h * p.group + (static_cast<int>(r) - token * p.group);
  const long long rows = static_cast<long long>(p.T) * p.Hq;
  float m = -INFINITY;
  bool nan = false;
  for (int s = lane; s < p.shares; s += 32) {
    const float ls = p.lse_part[s * rows + row];
    nan = nan || isnan(ls);
    m = fmaxf(m, ls);
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  if (__any_sync(0xffffffffu, nan)) m = NAN;
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  float sum = 0.f;
  const float* src = p.o_part + row * D + lane * WIDE;
#pragma unroll 4
  for (int s = first; s < p.shares; s += WARPS) {
    const float ls = p.lse_part[s * rows + row];
    if (ls == -INFINITY) continue;
    const float wgt = expf(ls - m);
    sum += wgt;
#pragma unroll
    for (int e = 0; e < PER; e += WIDE) {
      float v[WIDE];
      const float* at = src + s * rows * D + e * 32;
      if constexpr (WIDE == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(at);
      else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(at);
#pragma unroll
      for (int i = 0; i < WIDE; ++i) acc[e + i] = fmaf(wgt, v[i], acc[e + i]);
    }
  }
  if constexpr (WARPS > 1) {
    static_assert(WARPS == 8, "a block's warps share its row");
#pragma unroll
    for (int e = 0; e < PER; ++e) s_acc[warp][e / WIDE * 32 * WIDE + lane * WIDE + e % WIDE] = acc[e];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += s_sum[w];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int e = threadIdx.x; e < D; e += 256) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += s_acc[w][e];
      p.o[row * D + e] = __float2bfloat16_rn(v * inv);
    }
  } else {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < PER; e += WIDE) {
      uint32_t w[WIDE / 2];
#pragma unroll
      for (int i = 0; i < WIDE / 2; ++i) w[i] = pack_bf16x2(acc[e + 2 * i] * inv, acc[e + 2 * i + 1] * inv);
      __nv_bfloat16* at = p.o + row * D + lane * WIDE + e * 32;
      if constexpr (WIDE == 4) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(at) = w[0];
    }
  }
  if (first == 0 && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

// Rows from which on each has a warp and not a block.
constexpr unsigned kManyRows = 8192;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Partial outputs and their LSE of `shares` shares.
size_t paged_bytes(int T, int Hq, int d, int shares, size_t* lse_offset) {
  if (shares <= 1) return 0;
  const size_t rows = static_cast<size_t>(T) * Hq;
  const size_t o_bytes = align256(static_cast<size_t>(shares) * rows * d * 4);
  if (lse_offset) *lse_offset = o_bytes;
  return o_bytes + align256(static_cast<size_t>(shares) * rows * 4);
}

bool head_dim(int d) { return d == 64 || d == 128 || d == 256; }
bool page_tokens(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

}  // namespace

cudaError_t launch_paged_combine(int d, const PagedParams& p, cudaStream_t stream) {
  const unsigned rows = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hkv) *
                        static_cast<unsigned>(p.max_q) * static_cast<unsigned>(p.group);
  if (rows >= kManyRows) {
    const unsigned grid = rows / 8 + (rows % 8 != 0);
    return d == 64    ? chain_launch(paged_combine_kernel<64, 1>, grid, 256, 0, stream, 1, p)
           : d == 128 ? chain_launch(paged_combine_kernel<128, 1>, grid, 256, 0, stream, 1, p)
                      : chain_launch(paged_combine_kernel<256, 1>, grid, 256, 0, stream, 1, p);
  }
  return d == 64    ? chain_launch(paged_combine_kernel<64, 8>, rows, 256, 0, stream, 1, p)
         : d == 128 ? chain_launch(paged_combine_kernel<128, 8>, rows, 256, 0, stream, 1, p)
                    : chain_launch(paged_combine_kernel<256, 8>, rows, 256, 0, stream, 1, p);
}

namespace {

int paged_forward(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache,
                  const void* v_cache, const float* k_scale, const float* v_scale,
                  const int32_t* block_table, int table_stride, const int32_t* q_start,
                  const int32_t* kv_len, void* o, float* lse, int B, int T, int Hq, int Hkv,
                  int d, int num_pages, int page_size, int max_q, int max_kv, float scale,
                  int causal, int num_splits, void* workspace, size_t workspace_bytes,
                  int drop_load, unsigned long long wait_timeout_ns, void* stream) {
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_len || !o || !lse)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !head_dim(d)) return ATTN_ERR_INVALID_ARG;
  if (num_pages < 1 || table_stride < 1 || max_q < 1 || max_kv < 1) return ATTN_ERR_INVALID_ARG;
  if (!page_tokens(page_size)) return ATTN_ERR_INVALID_ARG;
  if (!q_start && T % B != 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return ATTN_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > kMaxKvSplits) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * Hkv > 0x7fffffffLL ||
      static_cast<long long>(T) * Hq > 0x7fffffffLL ||
      static_cast<long long>(table_stride) * page_size > (1LL << 30))
    return ATTN_ERR_INVALID_ARG;
  constexpr long long kMost = 1LL << 46;
  if (q_stride_t < 0 || (T > 1 && q_stride_t > kMost / T) || q_stride_h < 0 || (Hq > 1 && q_stride_h > kMost / Hq))
    return ATTN_ERR_INVALID_ARG;
  const int group = Hq / Hkv;
  max_q = std::min(max_q, q_start ? T : T / B);
  const long long rows = static_cast<long long>(max_q) * group;
  const int tile_rows = paged_rows(d, rows);
  const long long tiles = (rows + tile_rows - 1) / tile_rows;
  // blocks of the two launches for one sequence (each factor is below 2^31, as T * Hq is)
  if (std::max(tiles * Hkv * num_splits, rows * Hkv) > 0x7fffffffLL / B) return ATTN_ERR_INVALID_ARG;
  if (tile_rows < kPrefillRows && (Hkv > 65535 || B > 65535)) return ATTN_ERR_INVALID_ARG;  // its grid's y and z
  size_t lse_off = 0;
  const int cluster = paged_cluster(tile_rows, num_splits);
  const size_t need = paged_bytes(T, Hq, d, num_splits / cluster, &lse_off);
  if (need > 0 && (!workspace || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
  auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (off(q, 16) || off(k_cache, 16) || off(v_cache, 16) || off(k_scale, 4) || off(v_scale, 4) ||
      off(block_table, 4) || off(q_start, 4) || off(kv_len, 4) || off(o, 16) || off(lse, 4) ||
      (need > 0 && off(workspace, 256)))
    return ATTN_ERR_MISALIGNED;
  if ((T > 1 && q_stride_t % 8) || (Hq > 1 && q_stride_h % 8)) return ATTN_ERR_MISALIGNED;
  const size_t blocks = static_cast<size_t>(num_pages) * Hkv;
  const size_t out_rows = static_cast<size_t>(T) * Hq;
  struct Span {
    const void* p;
    size_t n;
  };
  const Span outs[3] = {{o, out_rows * d * 2}, {lse, out_rows * 4}, {need > 0 ? workspace : nullptr, need}};
  const Span ins[8] = {{q, static_cast<size_t>((T - 1LL) * q_stride_t + (Hq - 1LL) * q_stride_h + d) * 2},
                       {k_cache, blocks * page_size * d},
                       {v_cache, blocks * page_size * d},
                       {k_scale, blocks * 4},
                       {v_scale, blocks * 4},
                       {block_table, static_cast<size_t>(B) * table_stride * 4},
                       {q_start, (static_cast<size_t>(B) + 1) * 4},
                       {kv_len, static_cast<size_t>(B) * 4}};
  auto overlap = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + b.n && y < x + a.n;
  };
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return ATTN_ERR_ALIAS;
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return ATTN_ERR_ALIAS;
  }
  int sms = 0;
  unsigned int* status = nullptr;
  int rc = device_info(&sms, &status);
  if (rc != ATTN_OK) return rc;
  alignas(64) CUtensorMap tk, tv;
  if (tile_rows >= kPrefillRows || page_size != 16) {  // (the split-KV kernel copies pages of 16 without TMA)
    const int box = paged_box_rows(d, page_size);
    if ((rc = encode_pages(&tk, k_cache, static_cast<long long>(blocks), page_size, d, box)) != ATTN_OK) return rc;
    if ((rc = encode_pages(&tv, v_cache, static_cast<long long>(blocks), page_size, d, box)) != ATTN_OK) return rc;
  }
  PagedParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.qs_t = T > 1 ? q_stride_t : 0, p.qs_h = Hq > 1 ? q_stride_h : 0;
  p.k_cache = static_cast<const uint8_t*>(k_cache), p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale, p.v_scale = v_scale;
  p.table = block_table, p.q_start = q_start, p.kv_len = kv_len;
  p.o = static_cast<__nv_bfloat16*>(o), p.lse = lse;
  if (need > 0) {
    p.o_part = static_cast<float*>(workspace);
    p.lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + lse_off);
  }
  p.status = status;
  p.B = B, p.T = T, p.Hq = Hq, p.Hkv = Hkv, p.group = group;
  p.per_seq = T / B, p.group_inv = (65536 + group - 1) / group;
  p.table_stride = table_stride, p.num_pages = num_pages, p.page_size = page_size;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.max_q = max_q, p.tiles = static_cast<int>(tiles);
  p.splits = num_splits;
  p.cluster = cluster;
  p.shares = num_splits / cluster;
  if (tile_rows >= kPrefillRows && num_splits == 1)
    p.tail_tile = static_cast<int>(paged_tail(tiles * Hkv * B, sms, max_q, max_kv, causal != 0));
  const long long units = (static_cast<long long>(max_kv) + kPagedUnit - 1) / kPagedUnit;
  p.chunk = static_cast<int>(std::min<long long>((units + num_splits - 1) / num_splits * kPagedUnit, 1LL << 30));
  p.causal = causal != 0;
  p.wait_timeout_ns = wait_timeout_ns, p.drop_load = drop_load;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_paged(d, tile_rows, &tk, &tv, p, st);
  if (e == cudaSuccess && p.shares > 1) e = launch_paged_combine(d, p, st);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace ea51

using namespace ea51;

extern "C" {

size_t attn_fwd_fp8_paged_workspace_size(int T, int Hq, int Hkv, int d, int max_q, int num_splits) {
  if (T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !head_dim(d) || max_q < 1) return 0;
  if (num_splits < 1 || num_splits > kMaxKvSplits || static_cast<long long>(T) * Hq > 0x7fffffffLL) return 0;
  const long long rows = static_cast<long long>(std::min(max_q, T)) * (Hq / Hkv);
  return paged_bytes(T, Hq, d, num_splits / paged_cluster(paged_rows(d, rows), num_splits), nullptr);
}

int attn_fwd_fp8_paged_num_splits(int B, int Hq, int Hkv, int d, int page_size, int max_q,
                                  int max_kv, int num_sms) {
  if (!page_tokens(page_size)) return 1;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !head_dim(d) || max_q < 1 || max_kv < 1 || num_sms < 1)
    return 1;
  const long long rows = static_cast<long long>(max_q) * (Hq / Hkv);
  const int tile_rows = paged_rows(d, rows);
  const double ctas = static_cast<double>((rows + tile_rows - 1) / tile_rows) * B * Hkv;
  // Modelled run time in us, from measured parts (GB300); a turn is kPagedUnit keys of one block.
  // A batch's lengths are on the device: what is smallest is the product of its time if all are
  // max_kv and of that if they fill 0.35 of it, the longest among them.  Over 12 batches (3 to 32
  // sequences of 2048 to 16384 keys, each head dim), all of one length and of lengths from an
  // eighth on, the counts taken cost 9 % more than each's best, and 15 % with the full length
  // alone.
  const double partial = static_cast<double>(B) * max_q * Hq * d * 8.0 / 5e6;  // a split's output, out and back
  const bool long_tile = tile_rows >= kPrefillRows;
  // Rows of the matrix instruction that are not used cost the split-KV kernel little, two tiles of
  // eight a fifth.
  const double wide = tile_rows == 16 ? 1.2 : 1.0;
  const double alone = (d == 256 ? 2.2 : 1.1) * wide;  // a turn's latency; 1.4 times that with company
  const double bytes = 0.73 * d / 128.0 * wide;        // a turn's share of the multiprocessor's bandwidth
  const double resident = paged_blocks(d, tile_rows, page_size);
  double best = 0;
  int best_s = 1;
  for (int s = 1; s <= kMaxKvSplits; ++s) {
    const double turns = std::ceil(std::ceil(static_cast<double>(max_kv) / kPagedUnit) / s);
    const double per_sm = ctas * s / num_sms;
    double t;
    if (long_tile) {
      // A turn of the tcgen05 kernel takes 1.75 us at each head dim, to begin and end a block 10,
      // the merge in a cluster 6; clusters of 3 and 4 leave multiprocessors empty, and a last wave
      // in halves takes half a wave.  Measured over nine shapes (64 to 4096 queries of 8192 to
      // 32768 keys), the count taken was the fastest or within 2 % of it.
      const bool cluster = s > 1 && s <= kPrefillCluster;
      double queue = per_sm <= 1.0 ? 1.0 : 0.5 * (std::ceil(per_sm) + per_sm) * (cluster && s > 2 ? 1.08 : 1.0);
      if (s == 1 && paged_tail(static_cast<long long>(ctas), num_sms, max_q, max_kv, true) > 0)
        queue = std::min(queue, std::floor(per_sm) + 0.5);
      t = 4.0 + queue * (turns * 1.75 + 10.0 + (cluster ? 6.0 : 0.0)) + (s > kPrefillCluster ? 3.0 + partial * s : 0.0);
    } else {
      // Clusters want all their blocks at once (B=64 up to 16384 keys, 32/8 heads: 165 us in
      // clusters of 4 to 8, 133 with 9 to 12 splits and the merge kernel), and large ones do not
      // fill the groups of multiprocessors that each has to fit in (288 blocks of 304 in clusters
      // of 6: 54 us, 240 in clusters of 5: 36).
      t = 1.0;
      for (const double fill : {1.0, 0.35}) {
        if (fill < 1.0 && B == 1) continue;
        const double held = per_sm * fill, waves = held / resident;
        const bool crowded = s > 1 && s <= kPagedCluster && waves > (s > 4 ? 0.85 : 1.0);
        const double latency = turns * alone * (held > 1.0 ? 1.4 : 1.0);
        const double queue = waves > 1.0 ? 1.0 + (std::ceil(waves) / waves - 1.0) * (B > 1 ? 0.3 : 1.0) : 1.0;
        const double through = held * (turns * bytes + 2.0) * queue;  // (2 us of it to begin and end a block)
        t *= (s > kPagedCluster ? 11.0 + partial * s : 4.0) +
             (std::max(latency, through) + 0.1 * std::min(latency, through)) * (crowded ? 1.4 : 1.0);
      }
    }
    if (s == 1 || t < best) {
      best = t;
      best_s = s;
    }
  }
  return best_s;
}

int attn_fwd_fp8_paged(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache,
                       const void* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* block_table, int table_stride, const int32_t* q_start,
                       const int32_t* kv_len, void* o, float* lse, int B, int T, int Hq, int Hkv,
                       int d, int num_pages, int page_size, int max_q, int max_kv, float scale,
                       int causal, int num_splits, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return paged_forward(q, q_stride_t, q_stride_h, k_cache, v_cache, k_scale, v_scale, block_table, table_stride, q_start,
                       kv_len, o, lse, B, T, Hq, Hkv, d, num_pages, page_size, max_q, max_kv, scale, causal, num_splits,
                       workspace, workspace_bytes, -1, kWaitTimeoutNs, stream);
}

int attn_selftest_fwd_fp8_paged_dropped_load(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache, const void* v_cache, const float* k_scale,
    const float* v_scale, const int32_t* block_table, int table_stride, const int32_t* q_start, const int32_t* kv_len,
    void* o, float* lse, int B, int T, int Hq, int Hkv, int d, int num_pages, int page_size, int max_q, int max_kv,
    float scale, int causal, int num_splits, void* workspace, size_t workspace_bytes, int drop_load,
    unsigned int timeout_ms, void* stream) {
  if (drop_load < 0 || timeout_ms < 1 || timeout_ms > 10000) return ATTN_ERR_INVALID_ARG;
  return paged_forward(q, q_stride_t, q_stride_h, k_cache, v_cache, k_scale, v_scale, block_table, table_stride, q_start,
                       kv_len, o, lse, B, T, Hq, Hkv, d, num_pages, page_size, max_q, max_kv, scale, causal, num_splits,
                       workspace, workspace_bytes, drop_load, static_cast<unsigned long long>(timeout_ms) * 1000000ull,
                       stream);
}

}  // extern "C"

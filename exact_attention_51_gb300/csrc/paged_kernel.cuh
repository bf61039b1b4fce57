// Attention of a few query rows over a paged e4m3 cache (decoding, drafted
// tokens): one pass over the keys, bounded by reading them.
//
// A thread block takes the rows (query tokens x the heads of one key head's
// group, at most R = 8 * NT) of one sequence and one share of its keys.  The keys
// come in stages of 4 * KT through a ring in shared memory, with their pages' scales;
// four warps take KT of each stage's keys each, with a running maximum,
// sum and output of their own, which are merged at the end.
//
// Who fills the ring goes by the page size.  Pages of 32 tokens and more: a fifth warp, by TMA, at
// most eight copies a stage.  A copy's issue takes the warp that does it some 150 cycles of the
// 1300 that a turn computes, so the others do not: one sequence of 32768 keys in 64-token pages, 8
// heads of 128, one block a head, takes 216 us, and 264 with rings that they fill themselves.
// Pages of 16 tokens would need 16 copies a stage, more than that warp gets through (64 sequences
// of up to 16384 keys: 152 us); there each of the four copies its own keys with cp.async, 16 bytes
// a lane (SELF; 129 us; by TMA the same, but 12.7 us and 11.1 for nine sequences of up to 3001 keys
// of 64).
//
// Everything is computed transposed, so that the keys are the 16-wide side of
// the matrix instruction and the few query rows its 8-wide one:
//     S^T = K Q^T     (16 keys x 8 rows, over d)
//     O^T += V^T P^T  (16 elements of d x 8 rows, over keys)
// The e4m3 codes become fp16 in registers, which holds them exactly; Q is
// scaled by a power of two a row, so that fp16 holds bf16's digits, and P is
// fp16.  (mma.sync is enough here: 8 rows need 2 x 8 multiply-adds a byte read, a
// few percent of what it delivers, and its operands come from registers, where
// the codes are converted.)
//
// V's scales differ from block to block.  They are folded into the exponent,
//     p' = exp2(s + log2 vs - M),  O = sum p' v8 / l,  l = sum p' / vs,
// with M the running maximum of s + log2 vs: the largest contribution to O, not
// the largest weight, is what fp16's range is centred on, and one matrix
// product accumulates blocks of any scales.  (p' leaves fp32's normal range 2^-133 below M, and its key l:
// a weight that matters only where V's scales differ by more than 2^100.)
//
// P is rounded to fp16, by up to 2^-11 of each weight, because two parts of P would be twice the
// products; l sums p' before that.  The results differ from those of a P in fp32 in 5 to 9 of 100
// bf16 elements, by a step (2^-11 to 2^-10 of O's norm), and are as far from 64 bits as those are:
// bf16's own rounding, 0.0016 to 0.0017 of the norm.
//
// Layout of the products in registers.  K: lane (g, c) = (lane / 4, lane % 4)
// reads 16 adjacent bytes (16c + 64j of the row), enough for four k-steps; Q's
// fragments are stored in that order of d.  V: ldmatrix.trans on pairs of
// bytes gives (d, d + 1) of two keys; one byte permutation makes the
// fragments of the even and of the odd d, which are rows 0-7 and 8-15 of the
// product.  P^T: the fp16 pairs of S^T, transposed by movmatrix.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_fwd_kernel.cuh"
#include "chain.cuh"
#include "paged.h"

namespace ea51 {

constexpr uint32_t kCodePagedKV = 0x141, kCodePagedEmpty = 0x142;

template <int D_, int NT_, bool SELF_>
struct PagedShape {
  static constexpr int D = D_, NT = NT_;
  static constexpr bool SELF = SELF_;
  static constexpr int R = 8 * NT;         // query rows
  static constexpr int WARPS = 4;          // that compute; the one that only copies is warp 4
  static constexpr int THREADS = (WARPS + (SELF ? 0 : 1)) * 32;
  static constexpr int KT = D == 256 ? 16 : 32;  // keys a warp takes at a time
  static constexpr int MT = KT / 16;
  static constexpr int BN = WARPS * KT;          // keys of a stage
  static constexpr int FILL = SELF ? KT : BN;    // keys that a warp fills
  static constexpr int GROUPS = FILL / 16;       // in sixteens, the smallest page
  static constexpr int FILLERS = SELF ? WARPS : 1;
  static constexpr int MIN_BLOCKS = paged_blocks(D, R, SELF ? 16 : 32);
  static constexpr int PW = D >= 128 ? 128 : 64;  // bytes of a swizzled panel's row
  static constexpr int PANELS = D / PW;
  static constexpr int TILE = BN * D;             // bytes of K or V in a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int STAGES = (MIN_BLOCKS == 3 ? 2 : 3) * (D == 64 ? 2 : 1);  // 64 or 96 KB
  // per stage [4][8]: -, K scale, log2 V scale, 1 / V scale of 16 keys; then which are hidden, by filler
  static constexpr int META = 160;
  static constexpr int OFF_Q = STAGES * STAGE;          // Q fragments
  static constexpr int OFF_META = OFF_Q + D * R * 2;
  static constexpr int OFF_ROWF = OFF_META + STAGES * META;
  static constexpr int OFF_BAR = OFF_ROWF + R * 4;      // full [STAGES][FILLERS], empty [STAGES]
  static constexpr int OFF_ABORT = OFF_BAR + (FILLERS + 1) * STAGES * 8;
  static constexpr int OFF_ML = OFF_ABORT + 8;  // [WARPS][R] maxima, then sums, then factors
  static constexpr int OFF_BLOCK = OFF_ML + 2 * WARPS * R * 4;  // [2][R] the block's maxima and sums
  static constexpr int SMEM = OFF_BLOCK + 2 * R * 4;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int OUT_PITCH = D + 8;  // floats; + 8: the pair stores of four rows miss each other's banks
  static constexpr int OFF_PART = WARPS * R * OUT_PITCH * 4;  // the block's merged output, behind the warps'
  static constexpr int MERGE_THREADS = THREADS, MERGE_BLOCKS = kPagedCluster, PART_PITCH = D;
  static_assert(OFF_PART % 16 == 0 && OFF_PART + R * D * 4 <= OFF_Q, "the merge reuses the ring");
  static_assert(BN / 16 <= 8 && OFF_BAR % 8 == 0 && OFF_META % 16 == 0, "stage layout");
  static constexpr bool Q_REGS = NT == 1 && D <= 128;  // Q's fragments stay in registers
};

struct PagedSeq {
  int q0, nq;   // first query token, query tokens
  int nk;       // keys (for the causal limit)
  int seen;     // keys that the page table holds
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b, bool report) {
  PagedSeq s;
  const int per = p.per_seq;
  s.q0 = p.q_start ? p.q_start[b] : b * per;
  const int q1 = p.q_start ? p.q_start[b + 1] : s.q0 + per;
  s.nk = max(p.kv_len[b], 0);
  const long long cap = static_cast<long long>(p.table_stride) * p.page_size;
  s.seen = static_cast<int>(min(static_cast<long long>(s.nk), cap));
  unsigned code = 0;
  if (s.seen < s.nk) code = kCodeBadPage;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.T) {
    s.q0 = 0;
    s.nq = 0;
    code = kCodeBadSequence;
  } else {
    s.nq = q1 - s.q0;
    if (s.nq > p.max_q) code = kCodeBadSequence;
  }
  if (report && code != 0) atomicCAS(p.status + 1, 0u, code);
  return s;
}

// Keys that row r (token r / group of the sequence) sees.
__device__ __forceinline__ int paged_limit(const PagedParams& p, const PagedSeq& s, int token) {
  if (!p.causal) return s.seen;
  return max(min(s.seen, token + s.nk - s.nq + 1), 0);
}

// ---- thread-block clusters
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this block's shared memory `addr` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
              : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Two e4m3 codes (the low or high half of a word) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
              : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16-byte asynchronous copy past L1; cp_async_arrive counts the arrival of all of a thread's copies so far.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Row (of 8) that the products' row i stands for.  With 128-byte rows, lanes
// of neighbouring i read the same 64-byte half of theirs, so they take rows
// that differ in bit 2, which the swizzle sends to the other half.
template <int PW>
__device__ __forceinline__ int paged_key(int i) {
  return PW == 128 ? (i >> 1) + 4 * (i & 1) : i;
}

// Address of 16-byte chunk `ch` of key `row` in a tile of KT keys, swizzled as TMA does.
template <int D, int KT>
__device__ __forceinline__ uint32_t paged_chunk(uint32_t tile, int row, int ch) {
  if constexpr (D == 64) return tile + row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
  return tile + (ch >> 3) * (KT * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

// fp16 pair with NaN replaced by zero; `nan` gets 1.0 in their place, 0 elsewhere.
__device__ __forceinline__ uint32_t split_nan(uint32_t x, uint32_t& nan) {
  const __half2 h = *reinterpret_cast<const __half2*>(&x);
  const __half2 n = __hneu2(h, h);
  nan = *reinterpret_cast<const uint32_t*>(&n);
  uint32_t keep = 0;
  if ((nan & 0xffffu) == 0) keep |= x & 0xffffu;
  if ((nan >> 16) == 0) keep |= x & 0xffff0000u;
  return keep;
}

// What a block's scores are multiplied by: its K scale (2^-60 at least) times the row's factor,
// which may be 0.  The smallest normal number on top, which others round away, keeps a masked -inf
// one however small they are.
__device__ __forceinline__ float score_factor(float k_scale, float row) { return fmaf(k_scale, row, 0x1p-126f); }

constexpr float kPagedGrow = 8.f;   // the offset moves when a term is past 2^8 of it
// p' is kept 2^7 larger: below 2^15 in all, and normal in fp16 down to 2^-21 of the offset
constexpr float kPagedShift = 7.f;

// Results of one row (and of four of its elements): final where the keys are in one
// share, else the share's part, for the merge kernel.
__device__ __forceinline__ void paged_store_lse(const PagedParams& p, int share, long long all_rows, long long row,
                                                float m, float sum) {
  const float lse = sum == 0.f ? -INFINITY : (m - kPagedShift + log2f(sum)) * kLn2;
  if (p.shares > 1) p.lse_part[share * all_rows + row] = lse;
  else p.lse[row] = lse;
}
template <int D>
__device__ __forceinline__ void paged_store(const PagedParams& p, int share, long long all_rows, long long row, int e,
                                            float4 v) {
  if (p.shares > 1) {
    *reinterpret_cast<float4*>(p.o_part + (share * all_rows + row) * D + e) = v;
  } else {
    uint2 w;
    w.x = pack_bf16x2(v.x, v.y);
    w.y = pack_bf16x2(v.z, v.w);
    *reinterpret_cast<uint2*>(p.o + row * D + e) = w;
  }
}

// Merge of a cluster's `active` first blocks (the others have left), each of which has its rows'
// maxima, sums and output (not divided) in its shared memory: the blocks share out the output's
// elements and read one another's memory.  The S::MERGE_THREADS first threads of every block call
// it; others pass the cluster's barrier as often.
template <typename S, typename Place>
__device__ __forceinline__ void paged_cluster_merge(const PagedParams& p, uint8_t* smem, uint32_t sbase, int share,
                                                    int rank, int active, int nrows, long long all_rows,
                                                    Place place) {
  constexpr int D = S::D, R = S::R;
  cluster_arrive();
  cluster_wait();
  for (int i = rank * S::MERGE_THREADS + threadIdx.x; i < nrows * (D / 4); i += active * S::MERGE_THREADS) {
    const int n = i / (D / 4), e = i % (D / 4) * 4;
    // all loads of another block's memory are on their way at once
    float ms[S::MERGE_BLOCKS], ls[S::MERGE_BLOCKS], m = -INFINITY;
    float4 v[S::MERGE_BLOCKS];
#pragma unroll
    for (int j = 0; j < S::MERGE_BLOCKS; ++j) {
      ms[j] = j < active ? cluster_ld(cluster_map(sbase + S::OFF_BLOCK + n * 4, j)) : -INFINITY;
      ls[j] = j < active ? cluster_ld(cluster_map(sbase + S::OFF_BLOCK + (R + n) * 4, j)) : 0.f;
      v[j] = j < active ? cluster_ld4(cluster_map(sbase + S::OFF_PART + (n * S::PART_PITCH + e) * 4, j))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < S::MERGE_BLOCKS; ++j) m = fmaxf(m, ms[j]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < S::MERGE_BLOCKS; ++j) {
      // (a row that saw no key of the block: factor 0, output 0)
      const float f = ms[j] == -INFINITY ? 0.f : ex2_approx(ms[j] - m);
      sum = fmaf(f, ls[j], sum);
      acc.x = fmaf(f, v[j].x, acc.x);
      acc.y = fmaf(f, v[j].y, acc.y);
      acc.z = fmaf(f, v[j].z, acc.z);
      acc.w = fmaf(f, v[j].w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    const long long row = place(n);
    paged_store<D>(p, share, all_rows, row, e, acc);
    if (e == 0) paged_store_lse(p, share, all_rows, row, m, sum);
  }
  cluster_arrive();  // no block leaves while another reads its memory
  cluster_wait();
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, S::MIN_BLOCKS)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ PagedParams p) {
  constexpr int D = S::D, NT = S::NT, R = S::R, KT = S::KT, MT = S::MT, STAGES = S::STAGES;
  constexpr int KSTEPS = D / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  chain_begin();
  // ---- which rows and keys
  // (the rows of a sequence and key head are one tile here: more of them are the tcgen05 kernel's)
  const int split = static_cast<int>(blockIdx.x), h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
  // The page numbers of the first PRO stages are on their way before the lengths are known: where
  // this share has keys at all, it begins at the first one.  Lane i has group i % GROUPS of stage i / GROUPS.
  constexpr int PRO = STAGES * S::GROUPS <= 32 ? STAGES : 32 / S::GROUPS;
  const bool fills = S::SELF || warp == S::WARPS;
  const int fill0 = S::SELF ? warp * KT : 0;  // first of the stage's keys that this warp fills
  const long long first = static_cast<long long>(split) * p.chunk;
  const int32_t* table = p.table + static_cast<long long>(b) * p.table_stride;
  const int early = lane / S::GROUPS * S::BN + fill0 + lane % S::GROUPS * 16;  // its first key, from `first` on
  int number0 = 0;
  if (fills && lane < PRO * S::GROUPS)
    number0 = table[min((first + early) >> p.page_shift, static_cast<long long>(p.table_stride - 1))];
  const PagedSeq seq = paged_seq(p, b, split == 0 && h == 0 && threadIdx.x == 0);
  const int nrows = min(seq.nq, p.max_q) * p.group;  // at most R
  if (nrows <= 0) return;
  auto token_of = [&](int r) { return p.group == 1 ? r : (r * p.group_inv) >> 16; };  // r / group, r and group up to 16
  const int lim_max = paged_limit(p, seq, token_of(nrows - 1));
  const int lim_min = paged_limit(p, seq, 0);
  const int t_begin = static_cast<int>(min(first, static_cast<long long>(lim_max)));
  const int t_end = split == p.splits - 1
                        ? lim_max
                        : static_cast<int>(min(first + p.chunk, static_cast<long long>(lim_max)));
  // row r's place in q, o and lse
  auto place = [&](int r) {
    const int token = token_of(r);
    return static_cast<long long>(seq.q0 + token) * p.Hq + h * p.group + (r - token * p.group);
  };
  const long long all_rows = static_cast<long long>(p.T) * p.Hq;
  // the cluster's partial result, the block in it
  const int share = split / p.cluster, rank = split - share * p.cluster;
  float* s_block = reinterpret_cast<float*>(smem + S::OFF_BLOCK);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + S::OFF_ABORT);
  if (t_begin >= t_end && p.splits > 1) {  // no key here for these rows
    // (in a cluster the others do without it; if there are none, block 0 goes on and writes the empty rows)
    if (p.cluster == 1)
      for (int n = threadIdx.x; n < nrows; n += S::THREADS) p.lse_part[share * all_rows + place(n)] = -INFINITY;
    if (p.cluster == 1 || rank > 0) return;
  }
  // blocks of the cluster that have keys: shares of a chunk each, from the first on (and the last
  // takes the rest)
  const long long shares_used = (static_cast<long long>(lim_max) + p.chunk - 1) / p.chunk;
  const int active = p.cluster == 1 ? 1 : max(1, static_cast<int>(min(shares_used, static_cast<long long>(p.cluster))));

  // ---- the ring
  auto full = [&](int st) { return sbase + S::OFF_BAR + 8u * static_cast<uint32_t>(S::SELF ? st * S::WARPS + warp : st); };
  auto empty = [&](int st) { return sbase + S::OFF_BAR + 8u * static_cast<uint32_t>(S::FILLERS * STAGES + st); };
  const Waiter w{abort_flag, p.status, p.wait_timeout_ns};
  const int n_stages = (t_end - t_begin + S::BN - 1) / S::BN;
  bool ok = true;
  int k = 0, st = 0;
  uint32_t phase = 0;
  if (threadIdx.x == 0) *abort_flag = 0u;
  if (fills && lane == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full(i), S::SELF ? 33 : 2);  // the copies' arrival (each lane's, if it copies) and the scales'
      if (!S::SELF) mbar_init(empty(i), S::WARPS);
    }
    fence_mbarrier_init();
  }
  __syncwarp();
  // This warp's rows of Q, whose loads are on their way before the ring's first fill.
  constexpr int QROWS = R / S::WARPS, QPART = (D + 127) / 128;
  uint2 q_raw[QROWS][QPART];
  if (warp < S::WARPS) {
#pragma unroll
    for (int i = 0; i < QROWS; ++i) {
      const int n = warp + i * S::WARPS, token = token_of(n);
      const __nv_bfloat16* src = p.q + (seq.q0 + token) * p.qs_t + (h * p.group + (n - token * p.group)) * p.qs_h;
#pragma unroll
      for (int j = 0; j < QPART; ++j) {
        const int grp = lane + 32 * j;
        q_raw[i][j] = n < nrows && grp < D / 4 ? *reinterpret_cast<const uint2*>(src + grp * 4) : make_uint2(0, 0);
      }
    }
  }
  // A filling warp's state: lane g < GROUPS has the page and the scales of its keys 16 g .. 16 g + 15.
  // -1: no key of these is wanted, -2: a bad page number.
  auto key_at = [&](int j) { return t_begin + j * S::BN + fill0 + 16 * lane; };
  auto page_of = [&](int key, int number) {
    if (key >= t_end) return -1;
    return number >= 0 && number < p.num_pages ? number : -2;
  };
  auto number_at = [&](int j) {
    return j < n_stages && lane < S::GROUPS && key_at(j) < t_end ? table[key_at(j) >> p.page_shift] : 0;
  };
  const int box_rows = S::SELF ? 16 : min(p.page_size, S::BN);
  const bool starts_box = lane < S::GROUPS && ((16 * lane) & (box_rows - 1)) == 0;
  int pg = -1, pg_next = -1;
  float ks = 1.f, vs = 1.f;
  auto scales = [&] {
    const long long at = static_cast<long long>(pg) * p.Hkv + h;
    ks = pg >= 0 ? p.k_scale[at] : 1.f;
    vs = pg >= 0 ? p.v_scale[at] : 1.f;
  };
  // Sixteen keys of a head are 16 * D bytes in a row; by cp.async, lane l copies bytes 16 l of each 512.
  // Where those go in the tile, but for the swizzle's bits that the copy's number sets:
  uint32_t lane_at;
  if constexpr (D == 64) lane_at = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
  else if constexpr (D == 128) lane_at = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
  else lane_at = ((lane >> 3) & 1) * (S::BN * 128) + (lane >> 4) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
  // Copies and scales of this warp's part of stage j, whose pages are in pg.
  auto fill = [&](int j, int slot) {
    const unsigned hidden = __ballot_sync(0xffffffffu, lane < S::GROUPS && pg == -2);
    if constexpr (S::SELF) {
#pragma unroll
      for (int i = 0; i < S::GROUPS; ++i) {
        const int from = __shfl_sync(0xffffffffu, pg, i);
        if (from < 0) continue;
        const long long at = (static_cast<long long>(from) * p.Hkv + h) * (16 * D) + lane * 16;  // (pages of 16)
        const uint32_t tile = sbase + slot * S::STAGE + (fill0 + 16 * i) * S::PW;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          uint32_t to;
          if constexpr (D == 64) to = tile + u * 512 + lane_at;
          else if constexpr (D == 128) to = tile + u * 512 + (lane_at ^ ((u & 1) << 6));
          else to = tile + u * 256 + (lane_at ^ ((2 * u & 7) << 4));
          cp_async16(to, p.k_cache + at + u * 512);
          cp_async16(to + S::TILE, p.v_cache + at + u * 512);
        }
      }
      cp_async_arrive(full(slot));
    } else {
      const bool mine = starts_box && pg >= 0;
      const uint32_t box = static_cast<uint32_t>(box_rows * S::PW);
      const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) mbar_arrive_expect_tx(full(slot), boxes * 2 * S::PANELS * box);
      __syncwarp();
      if (mine) {
        const uint32_t to = sbase + slot * S::STAGE + (fill0 + 16 * lane) * S::PW;
        const int row = key_at(j) & (p.page_size - 1);
        const int block = pg * p.Hkv + h;  // num_pages * Hkv fits
#pragma unroll
        for (int pn = 0; pn < S::PANELS; ++pn) {
          tma_load_3d(to + pn * S::BN * S::PW, &tm_k, full(slot), pn * S::PW, row, block);
          tma_load_3d(to + S::TILE + pn * S::BN * S::PW, &tm_v, full(slot), pn * S::PW, row, block);
        }
      }
    }
    if (pg == -2 && lane < S::GROUPS) atomicCAS(p.status + 1, 0u, kCodeBadPage);
    float* m = reinterpret_cast<float*>(smem + S::OFF_META + slot * S::META);
    if (lane < S::GROUPS) {
      // (clamped, so that a scale that was never set cannot give 0 * inf)
      const float v = fminf(fmaxf(vs, 0x1p-60f), 0x1p60f);
      m[8 + fill0 / 16 + lane] = fmaxf(ks, 0x1p-60f);
      m[16 + fill0 / 16 + lane] = __log2f(v);
      m[24 + fill0 / 16 + lane] = 1.f / v;
    }
    if (lane == 0) reinterpret_cast<unsigned*>(m)[32 + (S::SELF ? warp : 0)] = hidden;
    __syncwarp();
    // (a test hook: the stage that lacks this arrival never fills.  Leaving its copies out as well
    // would cost calls without the hook 2 %: 24 ragged sequences at d = 256 25.2 us for 24.7)
    if (lane == 0 && j != p.drop_load) mbar_arrive(full(slot));
  };
  // What the fill after stage j uses is on its way until then.
  auto advance = [&](int j) {
    pg = lane < S::GROUPS && j + 1 < n_stages ? page_of(key_at(j + 1), pg_next) : -1;
    scales();
    pg_next = number_at(j + 2);
  };
  int filled = 0;
  if (fills) {
    const int after = number_at(PRO);
    pg = lane < PRO * S::GROUPS ? page_of(t_begin + early, number0) : -1;
    scales();
    const int page0 = pg;
    const float ks0 = ks, vs0 = vs;
#pragma unroll
    for (int i = 0; i < PRO; ++i) {  // (the ring is empty)
      const int from = (i * S::GROUPS + lane) & 31;
      pg = __shfl_sync(0xffffffffu, page0, from);
      ks = __shfl_sync(0xffffffffu, ks0, from);
      vs = __shfl_sync(0xffffffffu, vs0, from);
      if (lane >= S::GROUPS) pg = -1;
      if (i < n_stages) fill(i, i);
    }
    filled = min(PRO, n_stages);
    pg_next = after;
    advance(PRO - 1);
    for (; filled < min(STAGES, n_stages); ++filled) {
      fill(filled, filled);
      advance(filled);
    }
    if (!S::SELF && lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
  }

  // ---- Q: a power of two a row brings its largest element to [1, 2); fp16 fragments
  float* rowf = reinterpret_cast<float*>(smem + S::OFF_ROWF);
  if (warp < S::WARPS) {
#pragma unroll
    for (int rq = 0; rq < QROWS; ++rq) {
      const int n = warp + rq * S::WARPS;
      float f[QPART][4];
      float amax = 0.f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < QPART; ++i) {
        const uint2 raw = q_raw[rq][i];
        f[i][0] = __uint_as_float(raw.x << 16);
        f[i][1] = __uint_as_float(raw.x & 0xffff0000u);
        f[i][2] = __uint_as_float(raw.y << 16);
        f[i][3] = __uint_as_float(raw.y & 0xffff0000u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          amax = fmaxf(amax, fabsf(f[i][e]));
          nan = nan || !(fabsf(f[i][e]) < INFINITY);
        }
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      nan = __any_sync(0xffffffffu, nan);
      int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      if (nan) ex = 0;
      ex = max(ex, -126);  // (a row of zeros or subnormals, which have fewer digits)
      const float down = __uint_as_float(static_cast<unsigned>(127 - min(ex, 126)) << 23);
      const float up = __uint_as_float(static_cast<unsigned>(127 + min(ex, 126)) << 23);
#pragma unroll
      for (int i = 0; i < QPART; ++i) {
        // elements 4 grp .. 4 grp + 3: k-step 4 (d / 64) + d % 16 / 4 of lane (n % 8, d % 64 / 16)
        const int grp = lane + 32 * i;
        if (grp < D / 4) {
          const int ks = (grp >> 4) * 4 + (grp & 3), cc = (grp >> 2) & 3;
          uint2 v;
          v.x = pack_f16x2(f[i][0] * down, f[i][1] * down);
          v.y = pack_f16x2(f[i][2] * down, f[i][3] * down);
          *reinterpret_cast<uint2*>(smem + S::OFF_Q + ((ks * NT + (n >> 3)) * 32 + (n & 7) * 4 + cc) * 8) = v;
        }
      }
      if (lane == 0) rowf[n] = up * p.scale_log2;
    }
  }
  __syncthreads();

  float rf[NT][2];
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = nt * 8 + 2 * c + e;
      rf[nt][e] = rowf[n];
      lim[nt][e] = n < nrows ? paged_limit(p, seq, token_of(n)) : lim_max;
    }
  const uint32_t qf = sbase + S::OFF_Q + lane * 8;
  uint2 qreg[S::Q_REGS ? KSTEPS : 1];
  if constexpr (S::Q_REGS) {
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks) qreg[ks] = lds64(qf + ks * 256);
  }

  float o[D / 16][NT][4];
  float mx[NT][2], l[NT][2];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

  // exp2 gets s * f + log2 vs + base, base = kPagedShift - mx (a large number until a row has
  // seen a key, so that the first one moves mx)
  float base[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) base[nt][0] = base[nt][1] = 1e30f;

  if (!S::SELF && warp == S::WARPS) {
    for (; filled < n_stages; ++filled) {
      ok = warp_wait_phase(empty(st), phase, w, kCodePagedEmpty);
      if (!ok) break;
      fill(filled, st);
      advance(filled);
      if (++st == STAGES) st = 0, phase ^= 1u;
    }
    // No copy is in flight when the block ends, whoever's wait gives up before the stage is used.
    // (A stage that a test leaves unfilled has its copies behind it by the time that a wait for it gives up.)
    for (int i = max(0, filled - STAGES); i < filled; ++i)
      if (i != p.drop_load) drain_phase(full(i % STAGES), static_cast<uint32_t>(i / STAGES) & 1u, w, kCodeDrain);
    __syncwarp();
  } else {
    for (; k < n_stages; ++k) {
      ok = warp_wait_phase(full(st), phase, w, kCodePagedKV);
      if (!ok) break;
      const uint32_t kb = sbase + st * S::STAGE, vb = kb + S::TILE;
      const int t0 = t_begin + k * S::BN + warp * KT;
      if (t0 < t_end) {  // (a warp may have none of the last stage's keys)

        // ---- S^T = K Q^T
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint4 lo[MT], hi[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int r = warp * KT + mt * 16 + paged_key<S::PW>(g);
            lo[mt] = lds128(paged_chunk<D, S::BN>(kb, r, 4 * j + c));
            hi[mt] = lds128(paged_chunk<D, S::BN>(kb, r + 8, 4 * j + c));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int kstep = j * 4 + q;
            uint2 qb[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              qb[nt] = S::Q_REGS ? qreg[S::Q_REGS ? kstep : 0] : lds64(qf + (kstep * NT + nt) * 256);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t x = q == 0 ? lo[mt].x : q == 1 ? lo[mt].y : q == 2 ? lo[mt].z : lo[mt].w;
              const uint32_t y = q == 0 ? hi[mt].x : q == 1 ? hi[mt].y : q == 2 ? hi[mt].z : hi[mt].w;
              const uint32_t a0 = e4m3_lo(x), a1 = e4m3_lo(y), a2 = e4m3_hi(x), a3 = e4m3_hi(y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(s[mt][nt], a0, a1, a2, a3, qb[nt].x, qb[nt].y);
            }
          }
        }

        // ---- masks (a masked score is -inf), scales
        const float* meta = reinterpret_cast<const float*>(smem + S::OFF_META + st * S::META);
        // bit mt: these keys are hidden
        const unsigned* hides = reinterpret_cast<const unsigned*>(meta) + 32;
        const unsigned hidden = S::SELF ? hides[warp] : hides[0] >> (warp * MT);
        const bool partial = t0 + KT > lim_min || t0 + KT > t_end || (hidden & ((1u << MT) - 1)) != 0;
        float ksm[MT], lv[MT], inv_vs[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          ksm[mt] = meta[8 + warp * MT + mt];
          lv[mt] = meta[16 + warp * MT + mt];
          inv_vs[mt] = meta[24 + warp * MT + mt];
          if (partial) {
            const int key = t0 + mt * 16 + paged_key<S::PW>(g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int t = key + (e >> 1) * 8;
                if (((hidden >> mt) & 1u) || t >= lim[nt][e & 1] || t >= t_end) s[mt][nt][e] = -INFINITY;
              }
          }
        }

        // ---- exponents; the running maximum moves only when one is past it by kPagedGrow
        float x[MT][NT][4];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float f0 = score_factor(ksm[mt], rf[nt][0]), f1 = score_factor(ksm[mt], rf[nt][1]);
            x[mt][nt][0] = fmaf(s[mt][nt][0], f0, lv[mt] + base[nt][0]);
            x[mt][nt][1] = fmaf(s[mt][nt][1], f1, lv[mt] + base[nt][1]);
            x[mt][nt][2] = fmaf(s[mt][nt][2], f0, lv[mt] + base[nt][0]);
            x[mt][nt][3] = fmaf(s[mt][nt][3], f1, lv[mt] + base[nt][1]);
            grow = grow || fmax3(fmaxf(x[mt][nt][0], x[mt][nt][1]), x[mt][nt][2], x[mt][nt][3]) > kPagedGrow + kPagedShift;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = mx[nt][e];
              float y[MT][2];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const float f = score_factor(ksm[mt], rf[nt][e]);
                y[mt][0] = fmaf(s[mt][nt][e], f, lv[mt]);
                y[mt][1] = fmaf(s[mt][nt][e + 2], f, lv[mt]);
                m = fmax3(m, y[mt][0], y[mt][1]);
              }
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              if (m > mx[nt][e]) {
                const float alpha = ex2_approx(mx[nt][e] - m);
                mx[nt][e] = m;
                base[nt][e] = kPagedShift - m;
                l[nt][e] *= alpha;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[i][nt][e] *= alpha, o[i][nt][e + 2] *= alpha;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  x[mt][nt][e] = y[mt][0] + base[nt][e];
                  x[mt][nt][e + 2] = y[mt][1] + base[nt][e];
                }
              }
            }
        }

        // ---- P, its sum, and P^T's fragments
        uint32_t pb[MT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float p0 = ex2_approx(x[mt][nt][0]), p1 = ex2_approx(x[mt][nt][1]);
            const float p2 = ex2_approx(x[mt][nt][2]), p3 = ex2_approx(x[mt][nt][3]);
            l[nt][0] = fmaf(p0 + p2, inv_vs[mt], l[nt][0]);
            l[nt][1] = fmaf(p1 + p3, inv_vs[mt], l[nt][1]);
            pb[mt][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
            pb[mt][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
          }

        // ---- masked keys must not reach O through 0 * NaN.  Keys that no row sees
        // (behind the end, hidden pages): their codes are cleared.  Keys that only
        // some rows see: NaN codes are counted in a product of their own.
        bool nan_step = false;
        if (partial) {
          bool found = false;
          for (int i = lane; i < KT * (D / 16); i += 32) {
            const int r = i / (D / 16);
            const uint32_t at = paged_chunk<D, S::BN>(vb, warp * KT + r, i % (D / 16));
            if (((hidden >> (r / 16)) & 1u) || t0 + r >= t_end) {
              st_shared_v4(at, 0, 0, 0, 0);
            } else if (t0 + r >= lim_min) {
              const uint4 v = lds128(at);
              found = found || (__vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                                __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu)) != 0;
            }
          }
          if constexpr (!S::SELF) fence_proxy_async_smem();  // before TMA refills what was cleared
          nan_step = __any_sync(0xffffffffu, found);
          __syncwarp();
        }

        // ---- O^T += V^T P^T
        const int vrow = warp * KT + ((lane >> 3) & 1) * 8 + paged_key<S::PW>(lane & 7);
        if (!nan_step) {
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t v[4];
              ldmatrix_x4_trans(paged_chunk<D, S::BN>(vb, mt * 16 + vrow, 2 * cc + (lane >> 4)), v);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = __byte_perm(v[i], 0, 0x3120);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a0 = e4m3_lo(v[2 * i]), a1 = e4m3_hi(v[2 * i]);
                const uint32_t a2 = e4m3_lo(v[2 * i + 1]), a3 = e4m3_hi(v[2 * i + 1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(o[2 * cc + i][nt], a0, a1, a2, a3, pb[mt][nt][0], pb[mt][nt][1]);
              }
            }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t see[NT][2];  // 1.0 where the row sees the key, laid out as P^T
            const int key = t0 + mt * 16 + paged_key<S::PW>(g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t = key + e * 8;
                const bool in = !((hidden >> mt) & 1u) && t < t_end;
                see[nt][e] = movmatrix_trans(pack_f16x2(in && t < lim[nt][0] ? 1.f : 0.f, in && t < lim[nt][1] ? 1.f : 0.f));
              }
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t v[4];
              ldmatrix_x4_trans(paged_chunk<D, S::BN>(vb, mt * 16 + vrow, 2 * cc + (lane >> 4)), v);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = __byte_perm(v[i], 0, 0x3120);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t n0, n1, n2, n3;
                const uint32_t a0 = split_nan(e4m3_lo(v[2 * i]), n0), a1 = split_nan(e4m3_hi(v[2 * i]), n1);
                const uint32_t a2 = split_nan(e4m3_lo(v[2 * i + 1]), n2), a3 = split_nan(e4m3_hi(v[2 * i + 1]), n3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_f16(o[2 * cc + i][nt], a0, a1, a2, a3, pb[mt][nt][0], pb[mt][nt][1]);
                  float hit[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(hit, n0, n1, n2, n3, see[nt][0], see[nt][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (hit[e] > 0.f) o[2 * cc + i][nt][e] = NAN;
                }
              }
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if constexpr (S::SELF) {
        if (filled < n_stages) {
          fill(filled, st);
          advance(filled);
          ++filled;
        }
      } else {
        if (lane == 0) mbar_arrive(empty(st));
      }
      if (++st == STAGES) st = 0, phase ^= 1u;
    }
  }
  if constexpr (S::SELF) cp_async_wait_all();

  // ---- merge the four warps (the ring is free once all are here)
  __syncthreads();
  if (*abort_flag) {
    // nothing is valid, but the cluster's barriers need every block
    if (p.cluster > 1) cluster_arrive(), cluster_wait(), cluster_arrive(), cluster_wait();
    return;
  }
  float* out = reinterpret_cast<float*>(smem) + warp * R * S::OUT_PITCH;
  float* s_m = reinterpret_cast<float*>(smem + S::OFF_ML);
  float* s_l = s_m + S::WARPS * R;
  if (warp < S::WARPS) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int n = nt * 8 + 2 * c + e;
        if (g == 0) {
          s_m[warp * R + n] = mx[nt][e];
          s_l[warp * R + n] = sum;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(out + n * S::OUT_PITCH + i * 16 + 2 * g) = make_float2(o[i][nt][e], o[i][nt][e + 2]);
      }
  }
  __syncthreads();
  if (threadIdx.x < nrows) {
    const int n = threadIdx.x;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < S::WARPS; ++i) m = fmaxf(m, s_m[i * R + n]);
    float f[S::WARPS], sum = 0.f;
#pragma unroll
    for (int i = 0; i < S::WARPS; ++i) {
      f[i] = s_m[i * R + n] == -INFINITY ? 0.f : ex2_approx(s_m[i * R + n] - m);
      sum += f[i] * s_l[i * R + n];
    }
    // only a sum of exactly 0 is a row without keys (one with a NaN keeps it)
    const float inv = p.cluster > 1 ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < S::WARPS; ++i) s_l[i * R + n] = f[i] * inv;
    if (p.cluster > 1) {
      s_block[n] = sum == 0.f ? -INFINITY : isnan(sum) ? sum : m;
      s_block[R + n] = sum;
    } else {
      paged_store_lse(p, share, all_rows, place(n), m, sum);
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem);
  for (int i = threadIdx.x; i < nrows * (D / 4); i += S::THREADS) {
    const int n = i / (D / 4), e = i % (D / 4) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < S::WARPS; ++j) {
      // (a warp without keys has factor 0 and zeros)
      const float f = s_l[j * R + n];
      const float4 v = *reinterpret_cast<const float4*>(all + (j * R + n) * S::OUT_PITCH + e);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    if (p.cluster > 1) *reinterpret_cast<float4*>(smem + S::OFF_PART + (n * D + e) * 4) = acc;
    else paged_store<D>(p, share, all_rows, place(n), e, acc);
  }
  if (p.cluster > 1)
    paged_cluster_merge<S>(p, smem, sbase, share, rank, active, nrows, all_rows, [&](int n) { return place(n); });
}

}  // namespace ea51

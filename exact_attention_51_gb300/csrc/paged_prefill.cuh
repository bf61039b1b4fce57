// Attention of many query rows over a paged e4m3 cache (prompts and their
// chunks): bounded by the tensor cores.
//
// A thread block takes NQ tiles of 128 rows (query tokens x the heads of one key
// head's group) of one sequence and streams the keys they see through shared
// memory once:
//
//   TMA warp      pages of K_j and V_j, as e4m3, into rings; the pages' scales into a
//                 ring beside them.
//   converters    two warps: V_j -> fp16 (exact) in the swizzled layout that the MMA reads,
//                 once for all NQ * 128 rows.
//   MMA warp      S = Q K_j^T into tensor memory, O += P V_j with P read from there.
//   softmax       one warpgroup a tile, one thread a row, as attn_fwd_kernel; the first
//                 thing it does is to lay out its Q rows.
//
// K is multiplied as it is stored (kind::f8f6f4): a row of Q, its largest element brought to [2^7,
// 2^8) by a power of two, is the sum of an e4m3 row and an e5m2 row, and the two products cost what
// one of 16 bits does. e4m3 takes the upper four of bf16's eight digits; what rounding to them
// leaves is at most 8 of bf16's steps, which e5m2's three digits hold.  So elements of 2^-6 and
// more are exact (2^-13 of the row's largest and more).  Below, e4m3's step is 2^-9 and leaves up to 2^-10,
// where e5m2's is 2^-13: off by 2^-14 at most, 2^-21 of the row's largest. (With e4m3 for the
// second part as well, its range would end 2^-17 below.)  P has no such range -- a flat tail behind
// one heavy key is 2^-20 of it -- so P V is fp16 and V is converted: K's conversion would cost as
// much again of the shared memory's time.  (P's rounding: see paged_kernel.cuh.)
//
// Measured (32/8 heads of 128, pages of 64): a block takes 1.75 us for 128 keys and 10 to begin
// and end; 2 x 2048 queries against 16384 keys 833 us (1240 TFLOP/s of 4 d flops a
// key and row; less where scales that differ from page to page move the offset more often), 4096 against 4096
// 144.  Of a block's beginning and end a clock showed, in cycles: sequence and lengths 1250,
// barriers and tensor memory 1200, Q read and laid out 5400, the first scores 1700, a tile's softmax
// 2250, the output 4800.  Two tiles of 128 rows take turns on the tensor cores, which ncu has busy for
// 55 % of the time: the rest is the softmax's chain, as in attn_fwd_kernel.
//
// The scales are applied where they differ: one K scale for 16 keys (the smallest page)
// multiplies their scores in the softmax, and V's is folded into the exponent (see paged_kernel.cuh,
// whose running offset is kept here too).
#pragma once
#include <cuda_fp16.h>

#include "paged_kernel.cuh"

namespace ea51 {

constexpr int kMetaDepth = 8;  // tiles whose scales are held: more than the two rings are ahead of the softmax

enum : uint32_t {
  kCodePrefillRaw = 0x151,   // TMA warp, for a free slot
  kCodePrefillConv = 0x152,  // converters, for a V tile or a free fp16 slot
  kCodePrefillQ = 0x153,
  kCodePrefillKV = 0x154,
  kCodePrefillP = 0x155,
  kCodePrefillS = 0x156,
  kCodePrefillO = 0x157,
};

template <int D_>
struct PrefillShape {
  static constexpr int D = D_;
  // d = 256: one tile of 128 rows and 64 keys a tile (S twice and O: 384 tensor-memory columns)
  static constexpr int NQ = D == 256 ? 1 : 2, NSB = D == 256 ? 2 : 1, BN = D == 256 ? 64 : 128;
  static constexpr int ROWS = NQ * BM;
  static constexpr int GROUPS = BN / 16;
  // slots of K and V as stored, and of V in fp16
  static constexpr int KS = D == 64 ? 4 : 3, VS = D == 64 ? 3 : 2, FS = D == 64 ? 4 : 2;
  // 8-bit tiles: panels of PW-byte rows, swizzled over PW bytes
  static constexpr int PW = D >= 128 ? 128 : 64, PANELS8 = D / PW, RAW_BYTES = BN * D, RAW_PANEL = BN * PW;
  static constexpr int Q_PANEL = BM * PW, Q_PART = BM * D, Q_BYTES = 2 * Q_PART;  // [part][panel][row]
  // fp16 tiles: panels of 64 elements
  static constexpr int KV_PANEL = BN * 128, KV_BYTES = BN * D * 2;
  static constexpr int KSTEPS_QK = D / 32, KSTEPS_PV = BN / 16;
  static constexpr int P_PIECES = BN == 128 ? 2 : 1;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NQ * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KS * RAW_BYTES;
  static constexpr int OFF_F = OFF_V + VS * RAW_BYTES;
  // per tile [4][8]: page, K scale, log2 V scale, 1 / V scale; hidden groups
  static constexpr int OFF_META = OFF_F + FS * KV_BYTES;
  static constexpr int META = 160;
  static constexpr int OFF_BAR = OFF_META + kMetaDepth * META;
  static constexpr int B_Q = 0;  // [NQ], four warps each
  static constexpr int B_VEMPTY = B_Q + NQ;                // two warps each, as B_FFULL
  static constexpr int B_FFULL = B_VEMPTY + VS;
  static constexpr int B_P = B_FFULL + FS;                 // [NQ][NSB][P_PIECES], four warps each
  static constexpr int B_KFULL = B_P + NQ * NSB * P_PIECES;  // from here on one arrival each
  static constexpr int B_KEMPTY = B_KFULL + KS;
  static constexpr int B_VFULL = B_KEMPTY + KS;
  static constexpr int B_FEMPTY = B_VFULL + VS;
  static constexpr int B_META = B_FEMPTY + FS;             // [kMetaDepth]
  static constexpr int B_S = B_META + kMetaDepth;          // [NQ][NSB]
  static constexpr int B_ODONE = B_S + NQ * NSB;           // [NQ]
  static constexpr int B_OFINAL = B_ODONE + NQ;
  static constexpr int B_DRAIN = B_OFINAL + NQ;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_TMEMSLOT = OFF_BAR + NBAR * 8;
  static constexpr int OFF_ABORT = OFF_TMEMSLOT + 4;
  static constexpr int OFF_NAN = OFF_ABORT + 4;
  static constexpr int OFF_TILE = OFF_NAN + 4;
  static constexpr int SMEM_ALLOC = OFF_TILE + 96 + 1024;
  // a cluster's merge: each row's output, maximum and sum, where the tiles were (rows padded by 16 bytes: the
  // threads of a warp write a row each)
  static constexpr int R = ROWS, MERGE_THREADS = NQ * 128, PART_PITCH = D + 4;
  static constexpr int MERGE_BLOCKS = kPrefillCluster;  // blocks whose parts it reads at once
  static constexpr int OFF_PART = 0, OFF_BLOCK = R * PART_PITCH * 4;
  static_assert(OFF_BLOCK + 2 * R * 4 <= OFF_META, "the merge's rows");
  __host__ __device__ static constexpr int s_col(int q, int b) { return (q * NSB + b) * BN; }
  __host__ __device__ static constexpr int o_col(int q) { return NQ * NSB * BN + q * D; }
  static constexpr int TMEM_COLS = 512;
  static constexpr int TMA_WARP = 4 * NQ, MMA_WARP = 4 * NQ + 1, CONV_WARP = 4 * NQ + 2;
  static constexpr int CONV_THREADS = 64;
  static constexpr int THREADS = (NQ + 1) * 128;
  // as attn_fwd_kernel: 384 threads launch with 168 registers each, 256 * 40 = 128 * 80
  static constexpr bool SPLIT_REGS = NQ == 2;
  static constexpr int REG_SOFTMAX = 208, REG_CONTROL = 88;
  static_assert(!SPLIT_REGS || 256 * (REG_SOFTMAX - 168) <= 128 * (168 - REG_CONTROL), "register split");
  static_assert(NQ * NSB * BN + NQ * D <= TMEM_COLS && SMEM_ALLOC <= 232448, "budgets");
  // A cluster's blocks wait for one another with their tensor memory in hand.  Two clusters that shared two
  // multiprocessors could wait for each other's; a multiprocessor's 228 KB hold one block of this kernel.
  static_assert(2 * SMEM_ALLOC > 228 * 1024, "one block on a multiprocessor");
  static_assert(Q_PART % 1024 == 0 && KV_BYTES % 1024 == 0 && RAW_BYTES % 1024 == 0 && OFF_BAR % 8 == 0, "alignment");
};

template <typename S>
struct PrefillTile {
  PagedSeq seq;
  int h, b;
  int split, splits;  // which of the shares of the keys
  int cluster;        // blocks of the cluster that share this tile (1: none do, or by way of the workspace)
  int row0, rows;     // first row of the block, rows of the sequence and key head
  int lo;             // first key tile
  int nkv[S::NQ];     // key tiles [lo, lo + nkv) of each row tile
  int n;              // the most of them
  int t_end;          // keys from here on are not this block's
  int lim_min;        // keys that every row of the block sees
};

// kind::f8f6f4 descriptor with e5m2 A (format 1) and e4m3 B, both K-major, and fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc_e5m2_e4m3_f32(int M, int N) { return idesc_e4m3_f32(M, N) | (1u << 7); }

// kind::f16 descriptor with fp16 A and B (format 0) and fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <typename S>
__device__ __forceinline__ bool prefill_tile(const PagedParams& p, PrefillTile<S>& t, bool report) {
  int cta = static_cast<int>(blockIdx.x);
  if (p.tail_tile > 0) {  // (one split: the last wave's tiles are shared by two blocks)
    const int past = cta - p.tail_tile;
    t.splits = t.cluster = past < 0 ? 1 : 2;
    t.split = past < 0 ? 0 : past & 1;
    if (past >= 0) cta = p.tail_tile + (past >> 1);
  } else {
    t.splits = p.splits, t.cluster = p.cluster;
    t.split = cta % p.splits;
    cta /= p.splits;
  }
  t.h = cta % p.Hkv;
  cta /= p.Hkv;
  t.b = cta % p.B;
  const int tile = p.tiles - 1 - cta / p.B;  // the longest rows of every sequence first
  t.seq = paged_seq(p, t.b, report && t.split == 0 && t.h == 0 && tile == 0);
  t.rows = min(t.seq.nq, p.max_q) * p.group;
  t.row0 = tile * S::ROWS;
  if (t.row0 >= t.rows) return false;
  const int last = min(t.row0 + S::ROWS, t.rows) - 1;
  const int lim_max = paged_limit(p, t.seq, last / p.group);
  t.lim_min = paged_limit(p, t.seq, t.row0 / p.group);
  // A cluster's blocks hold a multiprocessor each until its last one is done: they share out the
  // keys that these rows see.  (Shares of a workspace are the same for all rows.)
  const int chunk = t.cluster > 1 ? max(1, (lim_max + S::BN * t.cluster - 1) / (S::BN * t.cluster)) * S::BN : p.chunk;
  const long long first = static_cast<long long>(t.split) * chunk;
  const int t_begin = static_cast<int>(min(first, static_cast<long long>(lim_max)));
  t.t_end = t.split == t.splits - 1 ? lim_max : static_cast<int>(min(first + chunk, static_cast<long long>(lim_max)));
  t.lo = t_begin / S::BN;  // a multiple of BN, or past every key
  t.n = 0;
#pragma unroll
  for (int q = 0; q < S::NQ; ++q) {
    const int r0 = t.row0 + q * BM;
    t.nkv[q] = 0;
    if (r0 < t.rows && t_begin < t.t_end) {
      const int lim = min(paged_limit(p, t.seq, (min(r0 + BM, t.rows) - 1) / p.group), t.t_end);
      t.nkv[q] = max(0, (lim + S::BN - 1) / S::BN - t.lo);
    }
    t.n = max(t.n, t.nkv[q]);
  }
  return true;
}

// The whole warp: lane g < GROUPS has the page and scales of keys 16 g .. 16 g + 15 of a tile.
template <typename S, typename Begin>
__device__ void prefill_load(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const PagedParams& p,
                             const PrefillTile<S>& t, uint8_t* smem, uint32_t sbase, Waiter w, Begin&& begin) {
  const int lane = threadIdx.x & 31;
  const uint32_t bar0 = sbase + S::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int32_t* table = p.table + static_cast<long long>(t.b) * p.table_stride;
  const int box_rows = min(p.page_size, S::BN);
  auto page_at = [&](int j) {
    const int key = (t.lo + j) * S::BN + 16 * lane;
    if (j >= t.n || lane >= S::GROUPS || key >= t.t_end) return -1;
    const int pg = table[key >> p.page_shift];
    return pg >= 0 && pg < p.num_pages ? pg : -2;
  };
  float ks = 1.f, vs = 1.f;
  auto scales = [&](int pg) {
    if (pg >= 0) {
      const long long at = static_cast<long long>(pg) * p.Hkv + t.h;
      ks = p.k_scale[at];
      vs = p.v_scale[at];
    } else {
      ks = vs = 1.f;
      if (pg == -2) atomicCAS(p.status + 1, 0u, kCodeBadPage);
    }
  };
  int pg = page_at(0);
  scales(pg);
  int pg_next = page_at(1);
  const bool starts_box = lane < S::GROUPS && (16 * lane) % box_rows == 0;
  begin();
  int issued[2] = {0, 0};  // tiles of K and of V
  bool ok = true;
  for (int j = 0; j < t.n && ok; ++j) {
    const bool mine = starts_box && pg >= 0;
    const uint32_t box = static_cast<uint32_t>(box_rows * S::PW);
    const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      constexpr int kSlots[2] = {S::KS, S::VS}, kFull[2] = {S::B_KFULL, S::B_VFULL}, kEmpty[2] = {S::B_KEMPTY, S::B_VEMPTY},
                    kOff[2] = {S::OFF_K, S::OFF_V};
      const int st = j % kSlots[kv];
      ok = warp_wait_phase(bar(kEmpty[kv] + st), (static_cast<uint32_t>(j / kSlots[kv]) & 1u) ^ 1u, w, kCodePrefillRaw);
      if (!ok) break;
      if (kv == 0) {
        float* m = reinterpret_cast<float*>(smem + S::OFF_META + (j % kMetaDepth) * S::META);
        const unsigned hidden = __ballot_sync(0xffffffffu, pg == -2);
        if (lane < 8) {
          const float v = fminf(fmaxf(vs, 0x1p-60f), 0x1p60f);
          reinterpret_cast<int*>(m)[lane] = pg;
          m[8 + lane] = fmaxf(ks, 0x1p-60f);
          m[16 + lane] = __log2f(v);
          m[24 + lane] = 1.f / v;
          if (lane == 0) reinterpret_cast<unsigned*>(m)[32] = hidden;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::B_META + j % kMetaDepth));
      }
      issued[kv] = j + 1;
      if (2 * j + kv == p.drop_load) continue;  // test hook: this slot never fills
      if (lane == 0) mbar_arrive_expect_tx(bar(kFull[kv] + st), boxes * S::PANELS8 * box);
      __syncwarp();
      if (mine) {
        const uint32_t dst = sbase + kOff[kv] + st * S::RAW_BYTES + 16 * lane * S::PW;
        const int row = ((t.lo + j) * S::BN + 16 * lane) & (p.page_size - 1);
#pragma unroll
        for (int pn = 0; pn < S::PANELS8; ++pn)
          tma_load_3d(dst + pn * S::RAW_PANEL, kv ? tm_v : tm_k, bar(kFull[kv] + st), pn * S::PW, row, pg * p.Hkv + t.h);
      }
    }
    if (!ok) break;
    pg = pg_next;
    scales(pg);
    pg_next = page_at(j + 2);
  }
  // no copy is in flight when the block ends, whoever's wait gives up before the tile is used
  for (int i = max(0, issued[0] - S::KS); i < issued[0]; ++i)
    if (2 * i != p.drop_load)
      drain_phase(bar(S::B_KFULL + i % S::KS), static_cast<uint32_t>(i / S::KS) & 1u, w, kCodeDrain);
  for (int i = max(0, issued[1] - S::VS); i < issued[1]; ++i)
    if (2 * i + 1 != p.drop_load)
      drain_phase(bar(S::B_VFULL + i % S::VS), static_cast<uint32_t>(i / S::VS) & 1u, w, kCodeDrain);
}

// Bytes of a word that are NaN codes, as 0xff each.
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Two warps: V_j as stored -> fp16.  A thread takes whole rows, so that eight lanes always
// access eight rows, whose chunks the swizzle spreads over the banks.
template <typename S>
__device__ void prefill_convert(const PagedParams& p, const PrefillTile<S>& t, uint8_t* smem, uint32_t sbase, Waiter w) {
  constexpr int D = S::D, CHUNKS = D / 16;
  const int tid = threadIdx.x - S::CONV_WARP * 32, lane = threadIdx.x & 31;
  const uint32_t bar0 = sbase + S::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* nan_flag = reinterpret_cast<volatile uint32_t*>(smem + S::OFF_NAN);
  for (int j = 0; j < t.n; ++j) {
    const int sv = j % S::VS, sf = j % S::FS;
    if (!warp_wait_phase(bar(S::B_VFULL + sv), static_cast<uint32_t>(j / S::VS) & 1u, w, kCodePrefillConv)) break;
    if (!warp_wait_phase(bar(S::B_FEMPTY + sf), (static_cast<uint32_t>(j / S::FS) & 1u) ^ 1u, w, kCodePrefillConv)) break;
    const volatile int* meta = reinterpret_cast<const volatile int*>(smem + S::OFF_META + (j % kMetaDepth) * S::META);
    const int key0 = (t.lo + j) * S::BN;
    // Codes of keys behind the end and of hidden pages are cleared.  Keys that only some
    // rows see must not reach the others through 0 * NaN: their NaN codes are cleared here
    // and put back by the rows that see them, at the end.
    const bool whole = key0 + S::BN <= t.t_end && key0 + S::BN <= t.lim_min && meta[32] == 0;
#pragma unroll 1
    for (int row = tid; row < S::BN; row += S::CONV_THREADS) {
      // the row's first chunk in either tile; chunk c is at that address with c exclusive-ored
      // into its chunk bits
      const uint32_t raw = paged_chunk<D, S::BN>(sbase + S::OFF_V + sv * S::RAW_BYTES, row, 0);
      const uint32_t out = sbase + S::OFF_F + sf * S::KV_BYTES + row * 128 + ((row & 7) << 4);
      auto read = [&](int c) { return lds128((raw ^ ((c & 7) << 4)) + (c >> 3) * S::RAW_PANEL); };
      auto write = [&](int c, const uint4& v) {
        const uint32_t at = (out ^ ((c & 3) << 5)) + (c >> 2) * S::KV_PANEL;
        st_shared_v4(at, e4m3_lo(v.x), e4m3_hi(v.x), e4m3_lo(v.y), e4m3_hi(v.y));
        st_shared_v4(at ^ 16, e4m3_lo(v.z), e4m3_hi(v.z), e4m3_lo(v.w), e4m3_hi(v.w));
      };
      if (whole) {
#pragma unroll
        for (int c = 0; c < CHUNKS; c += 4) {
          uint4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = read(c + u);
#pragma unroll
          for (int u = 0; u < 4; ++u) write(c + u, v[u]);
        }
      } else {
        const bool shown = key0 + row < t.t_end && meta[row >> 4] >= 0;
        const bool scan = key0 + row >= t.lim_min;
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) {
          uint4 v = read(c);
          if (!shown) v = make_uint4(0, 0, 0, 0);
          if (scan) {
            const uint4 bad = make_uint4(nan_codes(v.x), nan_codes(v.y), nan_codes(v.z), nan_codes(v.w));
            if (bad.x | bad.y | bad.z | bad.w) *nan_flag = 1u;
            v.x &= ~bad.x, v.y &= ~bad.y, v.z &= ~bad.z, v.w &= ~bad.w;
          }
          write(c, v);
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar(S::B_FFULL + sf));
      mbar_arrive(bar(S::B_VEMPTY + sv));
    }
  }
}

// One whole warp; see mma_role of attn_fwd_kernel.cuh for the order of the products.
template <typename S>
__device__ void prefill_mma(uint32_t tmem, uint32_t sbase, const PrefillTile<S>& t, Waiter w) {
  constexpr int NQ = S::NQ, NSB = S::NSB;
  constexpr uint32_t kQK[2] = {idesc_e4m3_f32(BM, S::BN), idesc_e5m2_e4m3_f32(BM, S::BN)};
  constexpr uint32_t kPV = idesc_f16_f32(BM, S::D, true);
  const uint32_t bar0 = sbase + S::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const uint32_t leader = elect_one();
  bool ok = true;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (t.nkv[q] > 0 && ok) ok = warp_wait_phase(bar(S::B_Q + q), 0u, w, kCodePrefillQ);
  auto wait_k = [&](int j) {
    return warp_wait_phase(bar(S::B_KFULL + j % S::KS), static_cast<uint32_t>(j / S::KS) & 1u, w, kCodePrefillKV);
  };
  auto wait_v = [&](int j) {
    return warp_wait_phase(bar(S::B_FFULL + j % S::FS), static_cast<uint32_t>(j / S::FS) & 1u, w, kCodePrefillKV);
  };
  auto release_k = [&](int j) { mma_commit(bar(S::B_KEMPTY + j % S::KS), leader); };
  auto release_v = [&](int j) { mma_commit(bar(S::B_FEMPTY + j % S::FS), leader); };
  auto issue_s = [&](int q, int b, int j) {
    constexpr int KPP = S::PW / 32;
    const uint64_t b0 = sdesc_swz<S::PW>(sbase + S::OFF_K + (j % S::KS) * S::RAW_BYTES, 16, 8 * S::PW);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint64_t a0 = sdesc_swz<S::PW>(sbase + S::OFF_Q + q * S::Q_BYTES + part * S::Q_PART, 16, 8 * S::PW);
#pragma unroll
      for (int k = 0; k < S::KSTEPS_QK; ++k) {
        const uint32_t ao = ((k / KPP) * S::Q_PANEL + (k % KPP) * 32) >> 4;
        const uint32_t bo = ((k / KPP) * S::RAW_PANEL + (k % KPP) * 32) >> 4;
        mma_ss_f8(tmem + S::s_col(q, b), a0 + ao, b0 + bo, part ? kQK[1] : kQK[0], part + k > 0 ? 1u : 0u, leader);
      }
    }
    mma_commit(bar(S::B_S + q * NSB + b), leader);
  };
  auto issue_pv = [&](int q, int b, int j, uint32_t pph) {
    const uint64_t b0 = sdesc_sw128(sbase + S::OFF_F + (j % S::FS) * S::KV_BYTES, S::KV_PANEL, 1024);
    constexpr int NP = S::P_PIECES, PER = S::KSTEPS_PV / NP;
#pragma unroll
    for (int h = 0; h < NP; ++h) {
      if (!warp_wait_phase(bar(S::B_P + (q * NSB + b) * NP + h), pph, w, kCodePrefillP)) return false;
      tc_fence_after_sync();
#pragma unroll
      for (int k = h * PER; k < (h + 1) * PER; ++k)
        mma_ts(tmem + S::o_col(q), tmem + S::s_col(q, b) + k * 8, b0 + ((k * 16 * 128) >> 4), kPV,
               (j > 0 || k > 0) ? 1u : 0u, leader);
    }
    mma_commit(bar(S::B_ODONE + q), leader);
    return true;
  };
  const int n = t.n;
  if (ok && n > 0) {
    if constexpr (NSB == 1) {
      ok = wait_k(0);
      if (ok) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          if (t.nkv[q] > 0) issue_s(q, 0, 0);
        release_k(0);
      }
      for (int j = 0; j < n && ok; ++j) {
        ok = wait_v(j);
        bool k_ready = false;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (!ok || j >= t.nkv[q]) continue;
          ok = issue_pv(q, 0, j, static_cast<uint32_t>(j) & 1u);
          if (!ok) break;
          if (j + 1 == t.nkv[q]) mma_commit(bar(S::B_OFINAL + q), leader);
          if (j + 1 < t.nkv[q]) {
            if (!k_ready) {
              ok = wait_k(j + 1);
              if (!ok) break;
              k_ready = true;
            }
            issue_s(q, 0, j + 1);
          }
        }
        if (!ok) break;
        release_v(j);
        if (k_ready) release_k(j + 1);
      }
    } else {
      for (int jj = 0; jj < 2 && jj < n && ok; ++jj) {
        ok = wait_k(jj);
        if (!ok) break;
        issue_s(0, jj, jj);
        release_k(jj);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int b = j & 1;
        ok = wait_v(j) && issue_pv(0, b, j, static_cast<uint32_t>(j >> 1) & 1u);
        if (!ok) break;
        if (j + 1 == n) mma_commit(bar(S::B_OFINAL), leader);
        release_v(j);
        if (j + 2 < n) {
          ok = wait_k(j + 2);
          if (!ok) break;
          issue_s(0, b, j + 2);
          release_k(j + 2);
        }
      }
    }
  }
  if (!ok) {
    mma_commit(bar(S::B_DRAIN), leader);
    drain_phase(bar(S::B_DRAIN), 0u, w, kCodeDrain);
  }
}

// P = exp2(s * ks * rf + (log2 vs - off)) of 32-column chunks [CH0, CH1) of a row as fp16 pairs, over the
// S columns already read; the scales are of 16 keys each (one page at most).  Returns the sum of P / vs.
template <int NCH, int CH0, int CH1>
__device__ __forceinline__ float prefill_exp(const uint32_t (&s)[NCH][32], float rf, const float* meta, float off,
                                             uint32_t s_t) {
  float total = 0.f;
#pragma unroll
  for (int ch = CH0; ch < CH1; ++ch) {
    const float2 ks = *reinterpret_cast<const float2*>(meta + 8 + ch * 2);
    const float2 lv = *reinterpret_cast<const float2*>(meta + 16 + ch * 2);
    const float2 iv = *reinterpret_cast<const float2*>(meta + 24 + ch * 2);
    uint32_t pk[16];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float a = (g ? lv.y : lv.x) - off, f = score_factor(g ? ks.y : ks.x, rf);
      const f32x2 ff = f2_pack(f, f), aa = f2_pack(a, a);
      f32x2 acc;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = g * 16 + 2 * e;
        const f32x2 x = f2_fma(f2_pack(__uint_as_float(s[ch][i]), __uint_as_float(s[ch][i + 1])), ff, aa);
        float t0, t1;
        f2_unpack(x, t0, t1);
        const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
        pk[g * 8 + e] = pack_f16x2(p0, p1);
        acc = e == 0 ? f2_pack(p0, p1) : f2_add(acc, f2_pack(p0, p1));
      }
      total = fmaf(f2_sum(acc), g ? iv.y : iv.x, total);
    }
    tmem_st_32x32b_x16(s_t + ch * 16, pk);
  }
  return total;
}

// Largest exponent of a row: per 16 keys the largest score, scaled (scales are positive).
template <int NCH>
__device__ __forceinline__ float prefill_max(const uint32_t (&s)[NCH][32], float rf, const float* meta) {
  float m = -INFINITY;
#pragma unroll
  for (int g = 0; g < 2 * NCH; ++g) {
    float a = __uint_as_float(s[g / 2][(g & 1) * 16]), b = __uint_as_float(s[g / 2][(g & 1) * 16 + 1]);
#pragma unroll
    for (int e = 2; e < 14; e += 4) {
      a = fmax3(a, __uint_as_float(s[g / 2][(g & 1) * 16 + e]), __uint_as_float(s[g / 2][(g & 1) * 16 + e + 1]));
      b = fmax3(b, __uint_as_float(s[g / 2][(g & 1) * 16 + e + 2]), __uint_as_float(s[g / 2][(g & 1) * 16 + e + 3]));
    }
    a = fmax3(a, __uint_as_float(s[g / 2][(g & 1) * 16 + 14]), __uint_as_float(s[g / 2][(g & 1) * 16 + 15]));
    m = fmaxf(m, fmaf(fmaxf(a, b), score_factor(meta[8 + g], rf), meta[16 + g]));
  }
  return m;
}

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Four fp32 values to e5m2 codes, nearest (b0 the lowest byte).
__device__ __forceinline__ uint32_t pack_e5m2x4(float b0, float b1, float b2, float b3) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(b0), "f"(b1), "f"(b2), "f"(b3));
  return r;
}

// A warp's 32 rows as it reads and writes them: a row is in LANES lanes of 16 bytes of bf16, and
// the I-th access has rows I * ROWS to (I + 1) * ROWS - 1.  (A row a thread touches 32 lines an
// access: with that a block of 128 keys, d = 128, took 14.2 us from its launch to the next one's,
// 11.6 this way.)
template <typename S>
struct PrefillRows {
  static constexpr int LANES = S::D / 8, ROWS = 32 / LANES, ACCESSES = LANES;
};

template <typename S>
struct PrefillQ {
  uint4 v[PrefillRows<S>::ACCESSES];
};

// Row `n` of the block in the tensors.
template <typename S>
__device__ __forceinline__ long long prefill_place(const PagedParams& p, const PrefillTile<S>& t, int n) {
  const int gr = t.row0 + n, token = gr / p.group;
  return static_cast<long long>(t.seq.q0 + token) * p.Hq + t.h * p.group + (gr - token * p.group);
}

// The loads of a warp's rows of Q, all on their way at once (zeros behind the last).
template <typename S>
__device__ __forceinline__ void prefill_fetch(int q, const PagedParams& p, const PrefillTile<S>& t, PrefillQ<S>& out) {
  using A = PrefillRows<S>;
  const int lane = threadIdx.x & 31, gr = t.row0 + q * BM + (threadIdx.x & 127);
  const int token = gr / p.group;
  const long long mine = gr < t.rows ? (t.seq.q0 + token) * p.qs_t + (t.h * p.group + (gr - token * p.group)) * p.qs_h : -1;
#pragma unroll
  for (int i = 0; i < A::ACCESSES; ++i) {
    const long long at = __shfl_sync(0xffffffffu, mine, i * A::ROWS + lane / A::LANES);
    out.v[i] = at >= 0 ? *reinterpret_cast<const uint4*>(p.q + at + lane % A::LANES * 8) : make_uint4(0, 0, 0, 0);
  }
}

// Lays out a warp's rows of Q, each with its largest element brought to [2^7, 2^8), as an e4m3 and
// an e5m2 row, and returns the factor of this thread's row's scores.
template <typename S>
__device__ __forceinline__ float prefill_lay_out(int q, uint32_t sbase, const PagedParams& p, const PrefillQ<S>& in) {
  using A = PrefillRows<S>;
  const int lane = threadIdx.x & 31;
  const uint32_t dst = sbase + S::OFF_Q + q * S::Q_BYTES;
  // bf16 magnitudes are ordered as their bits, infinities and NaN behind the rest
  uint32_t top[A::ACCESSES];
#pragma unroll
  for (int i = 0; i < A::ACCESSES; ++i) {
    const uint4 v = in.v[i];
    top[i] = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  }
#pragma unroll
  for (int m = A::LANES / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < A::ACCESSES; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], m));
  uint32_t mine = 0;  // this thread's row's
#pragma unroll
  for (int i = 0; i < A::ACCESSES; ++i) {
    top[i] = max(top[i] & 0xffffu, top[i] >> 16);
    const uint32_t other = __shfl_sync(0xffffffffu, top[i], lane % A::ROWS * A::LANES);
    if (lane / A::ROWS == i) mine = other;
  }
  // (down to -120, so that 2^7 times its reciprocal is a number; the bits of subnormals are all in range)
  auto exponent = [](uint32_t bits) {
    return bits >= 0x7f80u ? 0 : max(min(static_cast<int>(bits >> 7) - 127, 126), -120);
  };
#pragma unroll
  for (int i = 0; i < A::ACCESSES; ++i) {
    const uint32_t u[4] = {in.v[i].x, in.v[i].y, in.v[i].z, in.v[i].w};
    // a row with an infinity or NaN is NaN throughout, so that every score of it is, and a masked
    // one stays masked
    const float down =
        top[i] >= 0x7f80u ? NAN : __uint_as_float(static_cast<unsigned>(127 - exponent(top[i])) << 23) * 0x1p7f;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[2 * k] = __uint_as_float(u[2 * e + k] << 16) * down;
        x[2 * k + 1] = __uint_as_float(u[2 * e + k] & 0xffff0000u) * down;
      }
      hi[e] = pack_e4m3x4(x[0], x[1], x[2], x[3]);
      const uint32_t h01 = e4m3_lo(hi[e]), h23 = e4m3_hi(hi[e]);
      const float2 f01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
      const float2 f23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
      lo[e] = pack_e5m2x4(x[0] - f01.x, x[1] - f01.y, x[2] - f23.x, x[3] - f23.y);
    }
    const int r = (threadIdx.x & 96) + i * A::ROWS + lane / A::LANES;
    const uint32_t at = paged_chunk<S::D, BM>(dst, r, lane % A::LANES / 2) + (lane & 1) * 8;
    sts64(at, hi[0], hi[1]);
    sts64(at + S::Q_PART, lo[0], lo[1]);
  }
  return __uint_as_float(static_cast<unsigned>(127 + exponent(mine)) << 23) * 0x1p-7f * p.scale_log2;
}

// The same in a loop of four accesses, with the next four on their way, for d = 256: its 32
// accesses written out are much code for once a block and for one warp on each quarter of the
// multiprocessor.  Four waves of blocks of 128 keys take 55.9 us written out and 46.9 this way and with the
// output in a loop (d = 64 and 128 lose 0.6 and 3 by it).
template <typename S>
__device__ __forceinline__ float prefill_lay_out_loop(int q, uint32_t sbase, const PagedParams& p, const PrefillTile<S>& t) {
  using A = PrefillRows<S>;
  constexpr int G = 4;
  const int lane = threadIdx.x & 31, gr = t.row0 + q * BM + (threadIdx.x & 127);
  const int token = gr / p.group;
  const long long place = gr < t.rows ? (t.seq.q0 + token) * p.qs_t + (t.h * p.group + (gr - token * p.group)) * p.qs_h : -1;
  const uint32_t dst = sbase + S::OFF_Q + q * S::Q_BYTES;
  uint4 next[G];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const long long at = __shfl_sync(0xffffffffu, place, (i0 + k) * A::ROWS + lane / A::LANES);
      next[k] = at >= 0 ? *reinterpret_cast<const uint4*>(p.q + at + lane % A::LANES * 8) : make_uint4(0, 0, 0, 0);
    }
  };
  auto exponent = [](uint32_t bits) {
    return bits >= 0x7f80u ? 0 : max(min(static_cast<int>(bits >> 7) - 127, 126), -120);
  };
  uint32_t mine = 0;  // this thread's row's largest
  fetch(0);
#pragma unroll 1
  for (int i0 = 0; i0 < A::ACCESSES; i0 += G) {
    uint4 v[G];
    uint32_t top[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      v[k] = next[k];
      // bf16 magnitudes are ordered as their bits, infinities and NaN behind the rest
      top[k] = __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu), __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu));
    }
    if (i0 + G < A::ACCESSES) fetch(i0 + G);
#pragma unroll
    for (int m = A::LANES / 2; m > 0; m >>= 1)
#pragma unroll
      for (int k = 0; k < G; ++k) top[k] = __vmaxu2(top[k], __shfl_xor_sync(0xffffffffu, top[k], m));
#pragma unroll
    for (int k = 0; k < G; ++k) {
      top[k] = max(top[k] & 0xffffu, top[k] >> 16);
      const uint32_t other = __shfl_sync(0xffffffffu, top[k], lane % A::ROWS * A::LANES);
      if (lane / A::ROWS == i0 + k) mine = other;
    }
    uint32_t hi[G][2], lo[G][2];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      // (NaN throughout where there is an infinity or NaN, as prefill_lay_out)
      const float down =
          top[k] >= 0x7f80u ? NAN : __uint_as_float(static_cast<unsigned>(127 - exponent(top[k])) << 23) * 0x1p7f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[2 * j] = __uint_as_float(u[2 * e + j] << 16) * down;
          x[2 * j + 1] = __uint_as_float(u[2 * e + j] & 0xffff0000u) * down;
        }
        hi[k][e] = pack_e4m3x4(x[0], x[1], x[2], x[3]);
        const uint32_t h01 = e4m3_lo(hi[k][e]), h23 = e4m3_hi(hi[k][e]);
        const float2 f01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
        const float2 f23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
        lo[k][e] = pack_e5m2x4(x[0] - f01.x, x[1] - f01.y, x[2] - f23.x, x[3] - f23.y);
      }
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int r = (threadIdx.x & 96) + (i0 + k) * A::ROWS + lane / A::LANES;
      const uint32_t at = paged_chunk<S::D, BM>(dst, r, lane % A::LANES / 2) + (lane & 1) * 8;
      sts64(at, hi[k][0], hi[k][1]);
      sts64(at + S::Q_PART, lo[k][0], lo[k][1]);
    }
  }
  return __uint_as_float(static_cast<unsigned>(127 + exponent(mine)) << 23) * 0x1p-7f * p.scale_log2;
}

// What a softmax thread has of its row once the last product is in tensor memory.
template <typename S>
struct PrefillRow {
  float m = -INFINITY, l = 0.f;        // offset and sum; no key: 0
  bool has = false;                    // there is an output in tensor memory
  uint32_t nan_at[S::D / 32] = {};     // elements that a NaN of V makes one
};

template <typename S>
__device__ PrefillRow<S> prefill_softmax(int q, uint32_t tmem, uint8_t* smem, uint32_t sbase, const PrefillTile<S>& t,
                                         const PagedParams& p, const PrefillQ<S>& rows, Waiter w) {
  constexpr int D = S::D, BN = S::BN, NSB = S::NSB, NCH = BN / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t bar0 = sbase + S::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int n = t.nkv[q];
  PrefillRow<S> out;
  if (n == 0) return out;  // no key (of this share) for these rows

  float rf;
  if constexpr (S::D == 256) rf = prefill_lay_out_loop<S>(q, sbase, p, t);
  else rf = prefill_lay_out<S>(q, sbase, p, rows);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar(S::B_Q + q));

  const int token = min(t.row0 + q * BM + (warp & 3) * 32 + lane, t.rows - 1) / p.group;
  const int limit = min(paged_limit(p, t.seq, token), t.t_end), lo = t.lo;
  const uint32_t o_t = tmem + lane_base + S::o_col(q);
  float m_used = -INFINITY, l = 0.f;
  bool ok = true;
  for (int j = 0; j < n && ok; ++j) {
    const int b = NSB == 1 ? 0 : (j & 1);
    const uint32_t sph = static_cast<uint32_t>(NSB == 1 ? j : (j >> 1)) & 1u;
    ok = warp_wait_phase(bar(S::B_META + j % kMetaDepth), static_cast<uint32_t>(j / kMetaDepth) & 1u, w, kCodePrefillS) &&
         warp_wait_phase(bar(S::B_S + q * NSB + b), sph, w, kCodePrefillS);
    if (!ok) break;
    tc_fence_after_sync();
    const float* meta = reinterpret_cast<const float*>(smem + S::OFF_META + (j % kMetaDepth) * S::META);
    const uint32_t s_t = tmem + lane_base + S::s_col(q, b);
    uint32_t s[NCH][32];
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch) tmem_ld_32x32b_x32(s_t + ch * 32, s[ch]);
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch) tmem_ld_wait(s[ch]);
    const int lim = limit - (lo + j) * BN;
    const unsigned hidden = reinterpret_cast<const unsigned*>(meta)[32];
    if (__any_sync(0xffffffffu, lim < BN || hidden != 0)) {  // some row of the warp does not see the whole tile
#pragma unroll
      for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          s[ch][e] = ch * 32 + e < lim && !((hidden >> (ch * 2 + e / 16)) & 1u) ? s[ch][e] : 0xff800000u;
    }
    auto hand_over = [&](int part) {
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::B_P + (q * NSB + b) * S::P_PIECES + part));
    };
    const float mx = prefill_max<NCH>(s, rf, meta);
    if (j == 0) {
      m_used = mx;
    } else {
      const bool need = mx > m_used + kPagedGrow;
      if (__any_sync(0xffffffffu, need)) {
        ok = warp_wait_phase(bar(S::B_ODONE + q), static_cast<uint32_t>(j - 1) & 1u, w, kCodePrefillO);
        if (!ok) break;
        tc_fence_after_sync();
        const float alpha = need ? ex2_approx(m_used - mx) : 1.f;
        if (need) m_used = mx;
        l *= alpha;
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t ov[32];
          tmem_ld_32x32b_x32(o_t + ch * 32, ov);
          tmem_ld_wait(ov);
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tmem_st_32x32b_x32(o_t + ch * 32, ov);
        }
        tmem_st_wait();
      }
    }
    const float off = (m_used == -INFINITY ? 0.f : m_used) - kPagedShift;
    constexpr int CPP = NCH / S::P_PIECES;
    l += prefill_exp<NCH, 0, CPP>(s, rf, meta, off, s_t);
    hand_over(0);
    if constexpr (S::P_PIECES > 1) {
      l += prefill_exp<NCH, CPP, NCH>(s, rf, meta, off, s_t);
      hand_over(1);
    }
  }
  if (!ok || !warp_wait_phase(bar(S::B_OFINAL + q), 0u, w, kCodePrefillO)) return out;
  out.m = m_used, out.l = l, out.has = true;

  // V's NaN codes among the keys that only some rows see (cleared by the converters)
  if (*reinterpret_cast<volatile uint32_t*>(smem + S::OFF_NAN)) {
    const int32_t* table = p.table + static_cast<long long>(t.b) * p.table_stride;
    for (int key = max(t.lim_min, lo * BN); key < limit; ++key) {
      const int pg = table[key >> p.page_shift];
      if (pg < 0 || pg >= p.num_pages) continue;
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(
          p.v_cache + ((static_cast<long long>(pg) * p.Hkv + t.h) * p.page_size + (key & (p.page_size - 1))) * D);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        for (int e = 0; e < 8; ++e) {
          const uint32_t bad = nan_codes(codes[i * 8 + e]);
          const uint32_t bits = (bad & 1u) | ((bad >> 7) & 2u) | ((bad >> 14) & 4u) | ((bad >> 21) & 8u);
          out.nan_at[i] |= bits << (4 * e);
        }
    }
  }
  return out;
}

// A row's output times `factor`, 32 elements at a time, to use(chunk, values).
template <typename S, typename Use>
__device__ __forceinline__ void prefill_output(int q, uint32_t tmem, const PrefillRow<S>& row, float factor, Use&& use) {
  const uint32_t o_t = tmem + (static_cast<uint32_t>((threadIdx.x >> 5) & 3) * 32 << 16) + S::o_col(q);
#pragma unroll S::D == 256 ? 1 : S::D / 32
  for (int ch = 0; ch < S::D / 32; ++ch) {
    uint32_t marks = row.nan_at[0];
#pragma unroll
    for (int i = 1; i < S::D / 32; ++i) marks = ch == i ? row.nan_at[i] : marks;
    uint32_t ov[32];
    if (row.has) {  // (the same for a warp)
      tmem_ld_32x32b_x32(o_t + ch * 32, ov);
      tmem_ld_wait(ov);
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      // (a row that saw no key has P = 0 and O = 0, or, where V is NaN for others, nothing to show)
      const float v = row.l == 0.f ? 0.f : __uint_as_float(ov[e]) * factor;
      ov[e] = (marks >> e) & 1u ? 0x7fc00000u : __float_as_uint(v);
    }
    use(ch, ov);
  }
}

// The warp's results, or its parts to the workspace.
template <typename S>
__device__ __forceinline__ void prefill_store(int q, uint32_t tmem, uint32_t sbase, const PrefillTile<S>& t,
                                              const PagedParams& p, const PrefillRow<S>& row) {
  using A = PrefillRows<S>;
  const int lane = threadIdx.x & 31, n = threadIdx.x & 127;
  const bool valid = t.row0 + q * BM + n < t.rows;
  const long long mine = valid ? prefill_place<S>(p, t, q * BM + n) : -1;
  const long long all_rows = static_cast<long long>(p.T) * p.Hq;
  const float inv = row.l == 0.f ? 0.f : 1.f / row.l;
  if (valid) paged_store_lse(p, t.split, all_rows, mine, row.m, row.l);
  if (p.shares > 1) {
    prefill_output<S>(q, tmem, row, inv, [&](int ch, const uint32_t (&ov)[32]) {
      if (!valid || row.l == 0.f) return;  // (the merge passes over a part without keys)
      uint4* dst = reinterpret_cast<uint4*>(p.o_part + (t.split * all_rows + mine) * S::D + ch * 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
    });
    return;
  }
  // by way of the tile's Q, which its products are done with: chunk c of row n at c ^ (n % 8)
  const uint32_t base = sbase + S::OFF_Q + q * S::Q_BYTES;
  auto at = [&](int rr, int c) { return base + rr * S::D * 2 + ((c ^ (rr & 7)) << 4); };
  prefill_output<S>(q, tmem, row, inv, [&](int ch, const uint32_t (&ov)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_bf16x2(__uint_as_float(ov[8 * i + 2 * k]), __uint_as_float(ov[8 * i + 2 * k + 1]));
      st_shared_v4(at(n, ch * 4 + i), w[0], w[1], w[2], w[3]);
    }
  });
  __syncwarp();
#pragma unroll 4
  for (int i = 0; i < A::ACCESSES; ++i) {
    const int rr = i * A::ROWS + lane / A::LANES, c = lane % A::LANES;
    const long long to = __shfl_sync(0xffffffffu, mine, rr);
    const uint4 v = lds128(at((n & 96) + rr, c));
    if (to >= 0) *reinterpret_cast<uint4*>(p.o + to * S::D + c * 8) = v;
  }
}

// The row's part to this block's shared memory, for the cluster's merge; every role is done with
// the tiles there.
template <typename S>
__device__ __forceinline__ void prefill_offer(int q, uint32_t tmem, uint8_t* smem, const PrefillRow<S>& row) {
  const int n = q * BM + (threadIdx.x & 127);
  float* dst = reinterpret_cast<float*>(smem + S::OFF_PART) + n * S::PART_PITCH;
  prefill_output<S>(q, tmem, row, 1.f, [&](int ch, const uint32_t (&ov)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(dst + ch * 32 + 4 * i) = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
  });
  float* ml = reinterpret_cast<float*>(smem + S::OFF_BLOCK);
  ml[n] = row.l == 0.f ? -INFINITY : isnan(row.l) ? row.l : row.m;
  ml[S::R + n] = row.l;
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const PagedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  chain_begin();
  PrefillTile<S> t;
  if (!prefill_tile<S>(p, t, threadIdx.x == 0)) return;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + S::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::OFF_TMEMSLOT);
  // The warps that wait for copies have the caller's limit.  The softmax, which the abort flag
  // stops, has the usual one as a constant: its loop takes up to 7 % longer or shorter by what else
  // the compiler keeps in its registers (2 x 2048 queries against 16384 keys, d = 128: 837 us so,
  // 890 with the limit from the parameters).
  const Waiter w{abort_flag, p.status, p.wait_timeout_ns}, w_softmax{abort_flag, p.status};
  // for the epilogue, so that the softmax does not keep it in registers where those are short
  static_assert(sizeof(PrefillTile<S>) <= 96, "the tile's place");
  const PrefillTile<S>& tile = S::SPLIT_REGS ? *reinterpret_cast<const PrefillTile<S>*>(smem + S::OFF_TILE) : t;
  static_assert(S::NBAR <= S::MERGE_THREADS, "a thread a barrier");
  if (threadIdx.x < S::NBAR) {
    const int i = threadIdx.x, warps = i < S::B_VEMPTY ? 4 : i < S::B_P ? 2 : i < S::B_KFULL ? 4 : 1;
    mbar_init(sbase + S::OFF_BAR + 8u * i, warps);
    fence_mbarrier_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    *reinterpret_cast<volatile uint32_t*>(smem + S::OFF_NAN) = 0u;
    *reinterpret_cast<PrefillTile<S>*>(smem + S::OFF_TILE) = t;
  }
  if (warp == S::TMA_WARP && lane == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  // The block's barriers and tensor memory are there; what a role can load without them is on its
  // way by then.
  auto begin = [&] {
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    return *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  };
  if (warp < 4 * S::NQ) {
    const int q = warp >> 2;
    PrefillQ<S> rows;
    // (measured at d = 64 and 128, a block of 128 keys: 8.2 and 11.5 us before begin(), 8.3 and
    // 11.0 behind it)
    if constexpr (S::D == 64) prefill_fetch<S>(q, p, t, rows);
    const uint32_t tmem = begin();
    if constexpr (S::SPLIT_REGS) setmaxnreg_inc<S::REG_SOFTMAX>();
    if constexpr (S::D == 128) prefill_fetch<S>(q, p, t, rows);
    const PrefillRow<S> row = prefill_softmax<S>(q, tmem, smem, sbase, tile, p, rows, w_softmax);
    tc_fence_after_sync();
    if (tile.cluster == 1 && (row.has || tile.nkv[q] == 0))  // (not if a wait gave up)
      prefill_store<S>(q, tmem, sbase, tile, p, row);
    tc_fence_before_sync();
    __syncthreads();
    if (tile.cluster > 1) {
      tc_fence_after_sync();
      prefill_offer<S>(q, tmem, smem, row);
      tc_fence_before_sync();
      paged_cluster_merge<S>(p, smem, sbase, 0, tile.split, tile.cluster, min(S::ROWS, tile.rows - tile.row0),
                             static_cast<long long>(p.T) * p.Hq, [&](int n) { return prefill_place<S>(p, tile, n); });
    }
  } else {
    if constexpr (S::SPLIT_REGS) setmaxnreg_dec<S::REG_CONTROL>();
    uint32_t tmem = 0;
    if (warp == S::TMA_WARP) {
      prefill_load<S>(&tm_k, &tm_v, p, t, smem, sbase, w, begin);
    } else if (warp == S::MMA_WARP) {
      tmem_alloc(smem_addr(tmem_slot), S::TMEM_COLS);
      tmem_relinquish();
      tmem = begin();
      prefill_mma<S>(tmem, sbase, t, w);
    } else {
      begin();
      prefill_convert<S>(p, t, smem, sbase, w);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (t.cluster > 1) cluster_arrive(), cluster_wait(), cluster_arrive(), cluster_wait();  // as paged_cluster_merge
    if (warp == S::MMA_WARP) {
      tc_fence_after_sync();
      tmem_dealloc(tmem, S::TMEM_COLS);
    }
  }
}

}  // namespace ea51

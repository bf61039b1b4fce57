// Appending keys and values to the paged e4m3 cache: attn_paged_append_fp8 of
// include/attn_paged.h and its kernel.
//
// A run is the new tokens of one page.  A thread block takes one head of K or V and up to a
// page's worth of tokens (one, where the call has few), and the runs that begin among
// them in turn: it holds a run's (rotated) values in registers, reduces their
// largest magnitude, settles the block's scale 2^e and writes the codes; where
// the scale grows, it rewrites the codes of the tokens before the run.
//
// Why powers of two: moving a code from scale s to s * 2^j only changes its
// exponent, so a block whose scale grows token by token holds the same codes
// as one that was written at once, but for codes that fall below e4m3's
// normal range (2^-6 of the scale), which are rounded again.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_paged.h"
#include "chain.cuh"
#include "fwd_dispatch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace ea51 {
namespace {

constexpr int kMinExp = -60, kMaxExp = 60;
constexpr unsigned kCodeBadSlot = 0x201;

struct AppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long ks_t, ks_h, vs_t, vs_h;
  const int32_t* slots;
  const int32_t* pos;
  const uint64_t* phases;  // nullptr: no rotation
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  unsigned* index_status;
  float factor;
  int T, Hkv, rot, interleaved;
  int num_pages;
  int tokens_per_block;  // consecutive tokens whose runs one thread block takes in turn
};

// Smallest e in [kMinExp, kMaxExp] with amax <= 448 * 2^e, amax finite and
// >= 0: 448 = 1.75 * 2^8, so it is amax's exponent less 8, and one more where
// amax's significand is above 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
  const unsigned bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, a normal number
  return __uint_as_float(static_cast<unsigned>(e + 127) << 23);
}

// Four e4m3 codes times `ratio`, rounded to the nearest code.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t codes, float ratio) {
  float f[4];
  asm("{\n\t.reg .b16 lo, hi, a, b, c, d;\n\t.reg .b32 x, y;\n\t"
      "mov.b32 {lo, hi}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, lo;\n\tcvt.rn.f16x2.e4m3x2 y, hi;\n\t"
      "mov.b32 {a, b}, x;\n\tmov.b32 {c, d}, y;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\tcvt.f32.f16 %2, c;\n\tcvt.f32.f16 %3, d;\n\t}"
      : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
      : "r"(codes));
  return pack_e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// bf16 pair -> its two values.
__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}

// D: head dim.  PAGE: tokens a page.  A unit is 16 elements of one token; each
// thread holds two of a page's.  What bounds a prompt (14700 tokens of 8 heads of 128, 64 a page:
// 29.3 us, 3.1 TB/s; 16 a page: 27.4) is a block's chain of loads, barriers and some 25
// instructions an element, not the memory: rows fetched ahead for the blocks to come cost 2 us.
// Measured on it with a rotation of fewer instructions (rope.cuh): one unit a thread in 40 registers
// 32.9 us (512 threads to wait for at each barrier), two in 40 / 48 / 64 / 80 registers 29.5 / 27.1 / 27.0 /
// 30.6 (64: no spills, and 48 lose a tenth with pages of 16), four 35; the values of several heads in
// turn 33.
template <int D, int PAGE>
struct AppendShape {
  static constexpr int UNITS_PER_ROW = D / 16;
  static constexpr int UNITS = 2;
  static constexpr int BLOCK = PAGE * D / 16 / UNITS;  // 32 .. 1024
  static constexpr int MIN_BLOCKS = 1024 / BLOCK > 24 ? 24 : 1024 / BLOCK;
  static_assert(BLOCK <= 1024 && BLOCK % UNITS_PER_ROW == 0 && BLOCK >= 2 * PAGE, "append shape");
};

// The unit's elements: two groups of eight at `lo` and `hi` of the row.
// Rotated pairs in the half layout lie rot / 2 apart, so there a unit takes
// eight elements of each half; everywhere else it is 16 in a row.
__device__ __forceinline__ void unit_place(int u, int rot, bool split, int& lo, int& hi) {
  if (split && u < rot / 16) {
    lo = u * 8;
    hi = lo + rot / 2;
  } else {
    lo = u * 16;
    hi = lo + 8;
  }
}

// rot % 16 == 0: pairs are within the unit.
__device__ __forceinline__ void rotate_unit(float (&a)[16], int u, int pos, const AppendParams& p) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float c, s;
    rope_angle<false>(pos, p.phases[u * 8 + i], p.factor, c, s);
    if (p.interleaved) rope_turn(a[2 * i], a[2 * i + 1], c, s);
    else rope_turn(a[i], a[8 + i], c, s);
  }
}

// Any even rot: element e's partner is read from the row.
__device__ __forceinline__ float rotate_one(float x, const __nv_bfloat16* row, int e, int pos,
                                            const AppendParams& p) {
  if (e >= p.rot) return x;
  int pair, other;
  bool first;
  if (p.interleaved) {
    pair = e >> 1;
    first = (e & 1) == 0;
    other = e ^ 1;
  } else {
    first = e < p.rot / 2;
    pair = first ? e : e - p.rot / 2;
    other = first ? e + p.rot / 2 : pair;
  }
  float c, s;
  rope_angle<false>(pos, p.phases[pair], p.factor, c, s);
  const float o = __bfloat162float(row[other]);
  return first ? fmaf(x, c, -(o * s)) : fmaf(x, c, o * s);
}

// ANY: rotations of any even rot (else rot % 16 == 0).
template <int D, int PAGE, bool ANY>
__global__ void __launch_bounds__(AppendShape<D, PAGE>::BLOCK, ANY ? 1 : AppendShape<D, PAGE>::MIN_BLOCKS)
    attn_paged_append_kernel(const AppendParams p) {
  using S = AppendShape<D, PAGE>;
  constexpr int BLOCK = S::BLOCK, UPR = S::UNITS_PER_ROW, UNITS = S::UNITS;
  constexpr int WARPS = BLOCK / 32;
  constexpr int WORDS = 2 * PAGE / 32;
  __shared__ float s_amax[WARPS];
  __shared__ unsigned s_begin[WORDS], s_on[WORDS + 1];
  chain_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* src = is_v ? p.v + h * p.vs_h : p.k + h * p.ks_h;
  const long long st = is_v ? p.vs_t : p.ks_t;
  uint8_t* cache = is_v ? p.v_cache : p.k_cache;
  float* scales = is_v ? p.v_scale : p.k_scale;
  const bool rotate = !is_v && p.phases != nullptr;
  const bool split = rotate && !ANY && !p.interleaved;
  const long long limit = static_cast<long long>(p.num_pages) * PAGE;

  // The rows' way from HBM starts before the runs are known: a prompt's tokens are mostly one run.
  // (A block's own chain -- slots, rows, largest value, codes -- is what bounds this kernel: 3 us
  // of the prompt above.)
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int r = (tid + i * BLOCK) / UPR, u = (tid + i * BLOCK) % UPR;
    const int t = static_cast<int>(blockIdx.x) * p.tokens_per_block + r;
    if (r < p.tokens_per_block && t < p.T && u % 2 == 0)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(src + static_cast<long long>(t) * st + u * 16));
  }
  // which of this block's tokens begin a run, and which of them and of the page's worth behind
  // them go on with the run of the token before
  const int t0 = static_cast<int>(blockIdx.x) * p.tokens_per_block;
  const int n_tokens = min(p.T - t0, p.tokens_per_block);  // at most PAGE
  if (warp < WORDS) {
    bool begins = false, goes_on = false;
    if (tid < p.T - t0) {
      const int slot = p.slots[t0 + tid];
      const int before = t0 + tid > 0 ? p.slots[t0 + tid - 1] : -1;
      goes_on = slot > 0 && before == slot - 1 && slot % PAGE != 0;
      begins = slot >= 0 && !goes_on && tid < n_tokens;
      if (begins && slot >= limit) {
        atomicCAS(p.index_status, 0u, kCodeBadSlot);
        begins = false;
      }
    }
    const unsigned begin = __ballot_sync(0xffffffffu, begins), on = __ballot_sync(0xffffffffu, goes_on);
    if (lane == 0) s_begin[warp] = begin, s_on[warp] = on;
  }
  if (tid == 0) s_on[WORDS] = 0;
  __syncthreads();
#pragma unroll 1
  for (int next = 0; next < n_tokens; ++next) {
    // the next run's first token
    unsigned word = s_begin[next >> 5] >> (next & 31);
    while (word == 0 && (next | 31) + 1 < n_tokens) {
      next = (next | 31) + 1;
      word = s_begin[next >> 5];
    }
    if (word == 0) break;
    next += __ffs(word) - 1;
    const int t = t0 + next;
    const int slot = p.slots[t];
    const int page = slot / PAGE, off = slot % PAGE;
    // its length: 1 and the tokens behind that go on with it (at most a page in all)
    int end = next + 1;
#pragma unroll
    for (int w = 0; w <= PAGE / 32; ++w) {
      const unsigned stop = ~s_on[end >> 5] >> (end & 31);
      const int ones = stop ? __ffs(stop) - 1 : 32 - (end & 31);
      end += ones;
      if (stop) break;
    }
    const int len = end - next;

    float a[UNITS][16];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int r = (tid + i * BLOCK) / UPR, u = (tid + i * BLOCK) % UPR;
      if (r >= len) continue;
      const __nv_bfloat16* row = src + static_cast<long long>(t + r) * st;
      int lo, hi;
      unit_place(u, p.rot, split, lo, hi);
      const uint4 v0 = *reinterpret_cast<const uint4*>(row + lo), v1 = *reinterpret_cast<const uint4*>(row + hi);
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) unpack_bf16x2(w[j], a[i][2 * j], a[i][2 * j + 1]);
      if (rotate) {
        const int pos = p.pos[t + r];
        if constexpr (ANY) {
#pragma unroll
          for (int j = 0; j < 16; ++j) a[i][j] = rotate_one(a[i][j], row, u * 16 + j, pos, p);
        } else {
          if (u < p.rot / 16) rotate_unit(a[i], u, pos, p);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; j += 2) amax = fmax3(amax, fabsf(a[i][j]), fabsf(a[i][j + 1]));
    }
    if (amax == INFINITY) {  // rare: infinities become NaN, which the largest value passes over
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        if ((tid + i * BLOCK) / UPR >= len) continue;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          a[i][j] = fabsf(a[i][j]) < INFINITY ? a[i][j] : NAN;
          amax = fmaxf(amax, fabsf(a[i][j]));
        }
      }
    }
    // (not negative, so that their bits are ordered as they are)
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    const long long block = static_cast<long long>(page) * p.Hkv + h;
    const float had = off > 0 ? scales[block] : 0.f;
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) amax = fmaxf(amax, s_amax[w]);
    const float need = exp2_int(scale_exponent(amax));
    const float scale = fmaxf(need, had);  // a scale that was never set (0, NaN) counts as none
    uint8_t* codes = cache + block * (PAGE * D);
    if (had > 0.f && scale != had) {
      const float ratio = had / scale;
      for (int i = tid; i < off * D / 16; i += BLOCK) {
        uint4 w = reinterpret_cast<uint4*>(codes)[i];
        w.x = rescale_codes(w.x, ratio);
        w.y = rescale_codes(w.y, ratio);
        w.z = rescale_codes(w.z, ratio);
        w.w = rescale_codes(w.w, ratio);
        reinterpret_cast<uint4*>(codes)[i] = w;
      }
    }
    const float inv = 1.f / scale;  // a power of two: the product is exact
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int r = (tid + i * BLOCK) / UPR, u = (tid + i * BLOCK) % UPR;
      if (r >= len) continue;
      int lo, hi;
      unit_place(u, p.rot, split, lo, hi);
      uint8_t* row = codes + (off + r) * D;
      uint2 w;
      w.x = pack_e4m3x4(a[i][0] * inv, a[i][1] * inv, a[i][2] * inv, a[i][3] * inv);
      w.y = pack_e4m3x4(a[i][4] * inv, a[i][5] * inv, a[i][6] * inv, a[i][7] * inv);
      *reinterpret_cast<uint2*>(row + lo) = w;
      w.x = pack_e4m3x4(a[i][8] * inv, a[i][9] * inv, a[i][10] * inv, a[i][11] * inv);
      w.y = pack_e4m3x4(a[i][12] * inv, a[i][13] * inv, a[i][14] * inv, a[i][15] * inv);
      *reinterpret_cast<uint2*>(row + hi) = w;
    }
    if (tid == 0 && scale != had) scales[block] = scale;
    __syncthreads();  // the next run writes s_amax
  }
}

template <int D, int PAGE>
cudaError_t launch_append(AppendParams p, cudaStream_t stream) {
  // One token a block keeps a decoding step's latency at one run; where that would be far more
  // blocks than run at once (one without a run still takes its place), a block looks through
  // several tokens, up to a page's worth, in which a prompt has one or two runs.  Measured with
  // 2^18 threads in the grid and 2^20: 700 tokens of 8 heads in 16-token pages 4.6 us and 11.9, 69
  // x 32 tokens of 4 heads of 64 in pages of 128 6.1 and 8.3, 512 single tokens of 8 heads in
  // 64-token pages 20.3 and 21.6.
  constexpr long long kThreads = 1 << 18;
  const long long all = static_cast<long long>(p.T) * p.Hkv * 2 * AppendShape<D, PAGE>::BLOCK;
  p.tokens_per_block = 1;
  while (p.tokens_per_block < PAGE && all > kThreads * p.tokens_per_block) p.tokens_per_block *= 2;
  const dim3 grid(static_cast<unsigned>((p.T + p.tokens_per_block - 1) / p.tokens_per_block),
                  static_cast<unsigned>(p.Hkv), 2);
  constexpr unsigned kBlock = AppendShape<D, PAGE>::BLOCK;
  return p.rot % 16 == 0 ? chain_launch(attn_paged_append_kernel<D, PAGE, false>, grid, kBlock, 0, stream, 1, p)
                         : chain_launch(attn_paged_append_kernel<D, PAGE, true>, grid, kBlock, 0, stream, 1, p);
}

template <int D>
cudaError_t launch_append_d(const AppendParams& p, int page_size, cudaStream_t stream) {
  switch (page_size) {
    case 16: return launch_append<D, 16>(p, stream);
    case 32: return launch_append<D, 32>(p, stream);
    case 64: return launch_append<D, 64>(p, stream);
    default: return launch_append<D, 128>(p, stream);
  }
}

}  // namespace
}  // namespace ea51

extern "C" int attn_paged_append_fp8(const void* k, const void* v, int T, int Hkv, int d,
                                     int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
                                     int64_t v_stride_h, const int32_t* slots,
                                     const int32_t* positions, const uint64_t* phases, int rot_dim,
                                     int interleaved, float attention_factor, void* k_cache,
                                     void* v_cache, float* k_scale, float* v_scale, int num_pages,
                                     int page_size, void* stream) {
  using namespace ea51;
  if (T < 0 || Hkv < 1 || Hkv > 65535 || num_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return ATTN_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * Hkv > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_scale || !v_scale) return ATTN_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || !slots)) return ATTN_ERR_INVALID_ARG;
  if (phases) {
    if (T > 0 && !positions) return ATTN_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim > d || rot_dim % 2 != 0 || !std::isfinite(attention_factor))
      return ATTN_ERR_INVALID_ARG;
  }
  constexpr long long kMost = 1LL << 46;
  for (const int64_t s : {k_stride_t, v_stride_t})
    if (s < 0 || (T > 1 && s > kMost / T)) return ATTN_ERR_INVALID_ARG;
  for (const int64_t s : {k_stride_h, v_stride_h})
    if (s < 0 || (Hkv > 1 && s > kMost / Hkv)) return ATTN_ERR_INVALID_ARG;
  auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (off(k, 16) || off(v, 16) || off(k_cache, 16) || off(v_cache, 16) || off(k_scale, 4) ||
      off(v_scale, 4) || off(slots, 4) || off(positions, 4) || off(phases, 8))
    return ATTN_ERR_MISALIGNED;
  if ((T > 1 && (k_stride_t % 8 || v_stride_t % 8)) || (Hkv > 1 && (k_stride_h % 8 || v_stride_h % 8)))
    return ATTN_ERR_MISALIGNED;
  const size_t blocks = static_cast<size_t>(num_pages) * Hkv;
  const size_t cache_bytes = blocks * page_size * d, scale_bytes = blocks * 4;
  auto rows = [&](int64_t st, int64_t sh) {
    return T == 0 ? size_t{0} : static_cast<size_t>((T - 1LL) * st + (Hkv - 1LL) * sh + d) * 2;
  };
  struct Span {
    const void* p;
    size_t n;
  };
  const Span outs[4] = {{k_cache, cache_bytes}, {v_cache, cache_bytes}, {k_scale, scale_bytes}, {v_scale, scale_bytes}};
  const Span ins[5] = {{k, rows(k_stride_t, k_stride_h)},
                       {v, rows(v_stride_t, v_stride_h)},
                       {slots, static_cast<size_t>(T) * 4},
                       {phases ? positions : nullptr, static_cast<size_t>(T) * 4},
                       {phases, phases ? static_cast<size_t>(rot_dim) * 4 : 0}};
  auto overlap = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
  };
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return ATTN_ERR_ALIAS;
    for (const Span& in : ins)
      if (overlap(outs[i], in)) return ATTN_ERR_ALIAS;
  }
  int sms = 0;
  unsigned int* status = nullptr;
  const int rc = device_info(&sms, &status);
  if (rc != ATTN_OK) return rc;
  if (T == 0) return ATTN_OK;
  AppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.ks_t = k_stride_t, p.ks_h = k_stride_h, p.vs_t = v_stride_t, p.vs_h = v_stride_h;
  p.slots = slots;
  p.pos = positions;
  p.phases = phases;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.index_status = status + 1;
  p.factor = attention_factor;
  p.T = T, p.Hkv = Hkv, p.rot = phases ? rot_dim : 0, p.interleaved = interleaved != 0;
  p.num_pages = num_pages;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = d == 64    ? launch_append_d<64>(p, page_size, st)
                        : d == 128 ? launch_append_d<128>(p, page_size, st)
                                   : launch_append_d<256>(p, page_size, st);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

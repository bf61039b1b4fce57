// Rotary positions: the entry points of include/attn_rope.h and their kernel.
//
// A pass reads and writes every element once and computes one cos / sin pair
// for each position and frequency, so HBM bounds it once that pair (20 to 40
// instructions) is shared by several heads: a thread owns 2 * VEC elements of
// one position (VEC pairs) and walks over heads with its cos and sin in
// registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "attn_rope.h"
#include "chain.cuh"
#include "fwd_dispatch.h"
#include "rope.cuh"

namespace ea51 {
namespace {

struct RopeParams {
  const void* x;
  void* y;
  long long xs_b, xs_h, xs_n, ys_b, ys_h, ys_n;
  const int32_t* pos;
  long long pos_stride_b;
  int pos0;
  const uint64_t* phases;
  float factor;
  float sign;  // -1: the transpose
  int B, H, N, d, rot;
  int units;            // per head: rot / (2 VEC) rotated, then the copied ones
  int tokens_per_block;
  int heads_per_thread;
  int interleaved;
  int in_place;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// VEC elements in one access (16 bytes, or a single element).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

// Threads: tokens_per_block tokens x `units` units; blockIdx.y picks a group of
// heads_per_thread heads.  VEC = 16 bytes of elements where every row and pair half starts on 16 bytes,
// else 1.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) attn_rope_kernel(const RopeParams p) {
  chain_begin();
  const int tl = static_cast<int>(threadIdx.x) / p.units;
  const int u = static_cast<int>(threadIdx.x) - tl * p.units;
  if (tl >= p.tokens_per_block) return;
  const unsigned token = blockIdx.x * static_cast<unsigned>(p.tokens_per_block) + tl;
  if (token >= static_cast<unsigned>(p.B) * static_cast<unsigned>(p.N)) return;
  const int b = static_cast<int>(token / static_cast<unsigned>(p.N));
  const int n = static_cast<int>(token - static_cast<unsigned>(b) * static_cast<unsigned>(p.N));
  const int h0 = static_cast<int>(blockIdx.y) * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.H);
  const T* x = static_cast<const T*>(p.x) + b * p.xs_b + n * p.xs_n + h0 * p.xs_h;
  T* y = static_cast<T*>(p.y) + b * p.ys_b + n * p.ys_n + h0 * p.ys_h;
  using V = Pack<T, VEC>;
  const int rot_units = p.rot / (2 * VEC);
  if (u >= rot_units) {  // elements behind the rotated ones
    if (p.in_place) return;
    const int e = p.rot + (u - rot_units) * 2 * VEC;
    for (int h = h0; h < h1; ++h, x += p.xs_h, y += p.ys_h) {
      *reinterpret_cast<V*>(y + e) = *reinterpret_cast<const V*>(x + e);
      *reinterpret_cast<V*>(y + e + VEC) = *reinterpret_cast<const V*>(x + e + VEC);
    }
    return;
  }
  // pairs [u * VEC, u * VEC + VEC): half layout at e0 and e1 = e0 + rot / 2,
  // interleaved in the 2 * VEC elements from e0 on
  const int e0 = p.interleaved ? 2 * u * VEC : u * VEC;
  const int e1 = p.interleaved ? e0 + VEC : e0 + p.rot / 2;
  const int pos = p.pos ? p.pos[b * p.pos_stride_b + n] : p.pos0 + n;
  float c[VEC], s[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    rope_angle<sizeof(T) == 4>(pos, p.phases[u * VEC + i], p.factor, c[i], s[i]);
    s[i] *= p.sign;
  }
#pragma unroll 4
  for (int h = h0; h < h1; ++h, x += p.xs_h, y += p.ys_h) {
    V v0 = *reinterpret_cast<const V*>(x + e0), v1 = *reinterpret_cast<const V*>(x + e1);
    float f[2 * VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      f[i] = to_f32(v0.v[i]);
      f[VEC + i] = to_f32(v1.v[i]);
    }
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) rope_turn(f[2 * i], f[2 * i + 1], c[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) rope_turn(f[i], f[VEC + i], c[i], s[i]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v0.v[i] = from_f32<T>(f[i]);
      v1.v[i] = from_f32<T>(f[VEC + i]);
    }
    *reinterpret_cast<V*>(y + e0) = v0;
    *reinterpret_cast<V*>(y + e1) = v1;
  }
}

// Rows of whole 16-byte chunks whose pairs are not (rot / 2 not a multiple of a chunk's elements): a thread
// has one chunk of a row, and the half layout's partners come through shared memory, where they
// lie at any offset.  B=4 H=16 N=4096 d=128 bf16, rot = 118: 45.4 us, 75.7 element by element (its partners'
// 16-bit reads bound it); interleaved 36.6 and 76.5; fp32 d=256, rot = 246: 91 and 155.
template <typename T>
__global__ void __launch_bounds__(256) attn_rope_rows_kernel(const RopeParams p) {
  constexpr int VEC = 16 / sizeof(T);
  using V = Pack<T, VEC>;
  __shared__ V stage[2][256];
  chain_begin();
  const int tl = static_cast<int>(threadIdx.x) / p.units;
  const int u = static_cast<int>(threadIdx.x) - tl * p.units;
  const unsigned token = blockIdx.x * static_cast<unsigned>(p.tokens_per_block) + tl;
  // (threads without a row take part in the barriers)
  const bool active = tl < p.tokens_per_block && token < static_cast<unsigned>(p.B) * static_cast<unsigned>(p.N);
  const int b = static_cast<int>(token / static_cast<unsigned>(p.N));
  const int n = static_cast<int>(token - static_cast<unsigned>(b) * static_cast<unsigned>(p.N));
  const int h0 = static_cast<int>(blockIdx.y) * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.H);
  const int half = p.rot / 2, e0 = u * VEC;
  const T* x = static_cast<const T*>(p.x) + b * p.xs_b + n * p.xs_n + h0 * p.xs_h + e0;
  T* y = static_cast<T*>(p.y) + b * p.ys_b + n * p.ys_n + h0 * p.ys_h + e0;
  float c[VEC], s[VEC];
  if (active) {
    const int pos = p.pos ? p.pos[b * p.pos_stride_b + n] : p.pos0 + n;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int e = e0 + i;
      if (e >= p.rot) continue;
      const bool first = p.interleaved ? i % 2 == 0 : e < half;
      rope_angle<sizeof(T) == 4>(pos, p.phases[p.interleaved ? e / 2 : first ? e : e - half], p.factor, c[i], s[i]);
      s[i] *= first ? -p.sign : p.sign;
    }
  }
  V next;
  if (active) next = *reinterpret_cast<const V*>(x);
  for (int h = h0, buf = 0; h < h1; ++h, buf ^= 1) {
    V v = next;
    x += p.xs_h;
    if (active && h + 1 < h1) next = *reinterpret_cast<const V*>(x);
    T other[VEC];
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) other[i] = v.v[i ^ 1];
    } else {
      stage[buf][threadIdx.x] = v;
      __syncthreads();  // (once a head: before a buffer is written again, all have passed the next head's)
      const T* row = reinterpret_cast<const T*>(&stage[buf][threadIdx.x - u]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int e = e0 + i;
        if (active && e < p.rot) other[i] = row[e < half ? e + half : e - half];
      }
    }
    if (active) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (e0 + i < p.rot) v.v[i] = from_f32<T>(fmaf(to_f32(v.v[i]), c[i], to_f32(other[i]) * s[i]));
      *reinterpret_cast<V*>(y) = v;
    }
    y += p.ys_h;
  }
}

// heads that share a thread's cos and sin: as many as leave two blocks for
// each multiprocessor (measured against eight: B=4 H=16 N=4096 d=128 bf16 24.7 us, 23.8 with two; B=3 H=12
// N=1501 d=128 fp32 12.5 and 11.8)
int heads_per_thread(int H, long long blocks, int sms) {
  int hpt = 8;
  while (hpt > 1 && blocks * ((H + hpt - 1) / hpt) < 2LL * sms) hpt /= 2;
  while ((H + hpt - 1) / hpt > 65535) hpt *= 2;
  return hpt;
}

template <typename T>
cudaError_t launch_rope_rows(RopeParams p, int sms, cudaStream_t stream) {
  p.units = p.d / static_cast<int>(16 / sizeof(T));
  p.tokens_per_block = 256 / p.units;  // units <= 128: d <= 512
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const long long blocks = (tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  p.heads_per_thread = heads_per_thread(p.H, blocks, sms);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p.H + p.heads_per_thread - 1) / p.heads_per_thread));
  return chain_launch(attn_rope_rows_kernel<T>, grid, 256, 0, stream, 1, p);
}

template <typename T, int VEC>
cudaError_t launch_rope(RopeParams p, int sms, cudaStream_t stream) {
  p.units = p.d / (2 * VEC);
  p.tokens_per_block = 256 / p.units;  // units <= 256: d <= 512
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const long long blocks = (tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  p.heads_per_thread = heads_per_thread(p.H, blocks, sms);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p.H + p.heads_per_thread - 1) / p.heads_per_thread));
  return chain_launch(attn_rope_kernel<T, VEC>, grid, 256, 0, stream, 1, p);
}

template <typename T>
cudaError_t launch_rope_t(const RopeParams& p, int sms, cudaStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  auto ok = [&](long long stride) { return stride % VEC == 0; };
  const bool rows = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(p.y) % 16 == 0 && ok(p.xs_b) && ok(p.xs_h) &&
                    ok(p.xs_n) && ok(p.ys_b) && ok(p.ys_h) && ok(p.ys_n) && p.d % VEC == 0;
  if (!rows) return launch_rope<T, 1>(p, sms, stream);
  if (p.rot % (2 * VEC) == 0 && p.d % (2 * VEC) == 0) return launch_rope<T, VEC>(p, sms, stream);
  return launch_rope_rows<T>(p, sms, stream);
}

// Last element's offset + 1, of a [B, H, N, d] tensor with these strides.
long long extent(int B, int H, int N, int d, long long sb, long long sh, long long sn) {
  return (B - 1LL) * sb + (H - 1LL) * sh + (N - 1LL) * sn + d;
}

// Whether every element has a place of its own: ordered by stride, each dim
// steps over all that the smaller ones span.
bool distinct(int B, int H, int N, int d, long long sb, long long sh, long long sn) {
  std::pair<long long, long long> dims[3] = {{sb, B}, {sh, H}, {sn, N}};
  std::sort(dims, dims + 3);
  long long span = d;
  for (const auto& [stride, count] : dims) {
    if (count == 1) continue;
    if (stride < span) return false;
    span = stride * (count - 1) + span;
  }
  return true;
}

int rope(const void* x, void* y, int dtype, int B, int H, int N, int d, long long xs_b,
         long long xs_h, long long xs_n, long long ys_b, long long ys_h, long long ys_n,
         const int32_t* pos, long long pos_stride_b, int pos0, const uint64_t* phases, int rot,
         int interleaved, float factor, float sign, void* stream) {
  if (!x || !y || !phases) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_ROPE_BF16 && dtype != ATTN_ROPE_F16 && dtype != ATTN_ROPE_F32)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || N < 1 || d < 2 || d > 512 || d % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (rot < 2 || rot > d || rot % 2 != 0 || !std::isfinite(factor)) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (pos && pos_stride_b < 0) return ATTN_ERR_INVALID_ARG;
  if (!pos && pos0 > 0x7fffffff - (N - 1)) return ATTN_ERR_INVALID_ARG;
  // element offsets below 2^46 keep every product here in range
  constexpr long long kMost = 1LL << 46;
  for (const auto& [stride, count] :
       {std::pair<long long, long long>{xs_b, B}, {xs_h, H}, {xs_n, N}, {ys_b, B}, {ys_h, H}, {ys_n, N}})
    if (stride < 0 || (count > 1 && stride > kMost / count)) return ATTN_ERR_INVALID_ARG;
  if (pos && B > 1 && pos_stride_b > kMost / B) return ATTN_ERR_INVALID_ARG;
  if (!distinct(B, H, N, d, ys_b, ys_h, ys_n)) return ATTN_ERR_INVALID_ARG;
  const size_t es = dtype == ATTN_ROPE_F32 ? 4 : 2;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y);
  if (xa % es || ya % es || reinterpret_cast<uintptr_t>(phases) % 8 ||
      reinterpret_cast<uintptr_t>(pos) % 4)
    return ATTN_ERR_MISALIGNED;
  auto overlap = [](uintptr_t a, size_t na, uintptr_t b, size_t nb) { return a < b + nb && b < a + na; };
  const size_t xn = extent(B, H, N, d, xs_b, xs_h, xs_n) * es, yn = extent(B, H, N, d, ys_b, ys_h, ys_n) * es;
  auto same = [](long long a, long long b, int count) { return count == 1 || a == b; };
  const bool in_place = x == y && same(xs_b, ys_b, B) && same(xs_h, ys_h, H) && same(xs_n, ys_n, N);
  if (!in_place && overlap(xa, xn, ya, yn)) return ATTN_ERR_ALIAS;
  if (overlap(ya, yn, reinterpret_cast<uintptr_t>(phases), static_cast<size_t>(rot) * 4)) return ATTN_ERR_ALIAS;
  if (pos && overlap(ya, yn, reinterpret_cast<uintptr_t>(pos), ((B - 1) * pos_stride_b + N) * 4))
    return ATTN_ERR_ALIAS;
  int sms = 0;
  unsigned int* status = nullptr;
  const int rc = device_info(&sms, &status);
  if (rc != ATTN_OK) return rc;
  RopeParams p{};
  p.x = x;
  p.y = y;
  // a dim of one element never steps: its stride need not be aligned
  auto eff = [](long long stride, int count) { return count == 1 ? 0LL : stride; };
  p.xs_b = eff(xs_b, B), p.xs_h = eff(xs_h, H), p.xs_n = eff(xs_n, N);
  p.ys_b = eff(ys_b, B), p.ys_h = eff(ys_h, H), p.ys_n = eff(ys_n, N);
  p.pos = pos;
  p.pos_stride_b = pos_stride_b;
  p.pos0 = pos0;
  p.phases = phases;
  p.factor = factor;
  p.sign = sign;
  p.B = B, p.H = H, p.N = N, p.d = d, p.rot = rot;
  p.interleaved = interleaved != 0;
  p.in_place = in_place;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == ATTN_ROPE_BF16  ? launch_rope_t<__nv_bfloat16>(p, sms, st)
                        : dtype == ATTN_ROPE_F16 ? launch_rope_t<__half>(p, sms, st)
                                                 : launch_rope_t<float>(p, sms, st);
  return e == cudaSuccess ? ATTN_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace ea51

extern "C" {

int attn_rope_phases(uint64_t* phases, float* attention_factor, int rot_dim, double base,
                     int scaling, double factor, int original_positions, double beta_fast,
                     double beta_slow) {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (!phases || rot_dim < 2 || rot_dim > 512 || rot_dim % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 1.0) return ATTN_ERR_INVALID_ARG;
  if (scaling < ATTN_ROPE_NONE || scaling > ATTN_ROPE_YARN) return ATTN_ERR_INVALID_ARG;
  if (scaling != ATTN_ROPE_NONE && (!std::isfinite(factor) || factor < 1.0)) return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_NTK && rot_dim == 2) return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_YARN &&
      (original_positions < 1 || !std::isfinite(beta_fast) || !std::isfinite(beta_slow) || beta_fast <= beta_slow))
    return ATTN_ERR_INVALID_ARG;
  const double b = scaling == ATTN_ROPE_NTK
                       ? base * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2))
                       : base;
  if (!std::isfinite(b)) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == ATTN_ROPE_LINEAR) f /= factor;
    if (scaling == ATTN_ROPE_YARN) {
      const double turns = original_positions * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
      f = keep * f + (1.0 - keep) * f / factor;
    }
    phases[i] = static_cast<uint64_t>(std::ldexp(f / kTwoPi, 64));  // f <= 1: below a sixth of 2^64
  }
  if (attention_factor)
    *attention_factor = scaling == ATTN_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return ATTN_OK;
}

int attn_rope(const void* x, void* y, int dtype, int B, int H, int N, int d, int64_t x_stride_b,
              int64_t x_stride_h, int64_t x_stride_n, int64_t y_stride_b, int64_t y_stride_h,
              int64_t y_stride_n, const int32_t* positions, int64_t position_stride_b,
              int position0, const uint64_t* phases, int rot_dim, int interleaved,
              float attention_factor, void* stream) {
  return ea51::rope(x, y, dtype, B, H, N, d, x_stride_b, x_stride_h, x_stride_n, y_stride_b,
                    y_stride_h, y_stride_n, positions, position_stride_b, position0, phases,
                    rot_dim, interleaved, attention_factor, 1.f, stream);
}

int attn_rope_bwd(const void* dy, void* dx, int dtype, int B, int H, int N, int d,
                  int64_t dy_stride_b, int64_t dy_stride_h, int64_t dy_stride_n,
                  int64_t dx_stride_b, int64_t dx_stride_h, int64_t dx_stride_n,
                  const int32_t* positions, int64_t position_stride_b, int position0,
                  const uint64_t* phases, int rot_dim, int interleaved, float attention_factor,
                  void* stream) {
  return ea51::rope(dy, dx, dtype, B, H, N, d, dy_stride_b, dy_stride_h, dy_stride_n, dx_stride_b,
                    dx_stride_h, dx_stride_n, positions, position_stride_b, position0, phases,
                    rot_dim, interleaved, attention_factor, -1.f, stream);
}

}  // extern "C"

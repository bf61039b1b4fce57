// Kernel launch of attention over the paged cache for one head dim (all row
// tiles).  Included by one translation unit per head dim so that they compile
// in parallel.
#pragma once
#include <atomic>

#include "paged_kernel.cuh"
#include "paged_prefill.cuh"

namespace ea51 {

// The dynamic shared-memory opt-in of a kernel, once per device.
template <typename Kernel>
cudaError_t paged_configure(Kernel kern, int bytes, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (configured.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  configured.fetch_or(bit, std::memory_order_acq_rel);
  return cudaSuccess;
}

template <typename S>
cudaError_t launch_paged_shape(const CUtensorMap* tk, const CUtensorMap* tv, const PagedParams& p,
                               cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  auto kern = paged_attn_kernel<S>;
  const cudaError_t e = paged_configure(kern, S::SMEM_ALLOC, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.splits), static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B));
  return chain_launch(kern, grid, S::THREADS, S::SMEM_ALLOC, stream, static_cast<unsigned>(p.cluster), *tk, *tv, p);
}

template <int D>
cudaError_t launch_prefill(const CUtensorMap* tk, const CUtensorMap* tv, const PagedParams& p,
                           cudaStream_t stream) {
  using S = PrefillShape<D>;
  static std::atomic<unsigned long long> configured{0};
  auto kern = paged_prefill_kernel<S>;
  const cudaError_t e = paged_configure(kern, S::SMEM_ALLOC, configured);
  if (e != cudaSuccess) return e;
  const unsigned tiles = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.tiles) * static_cast<unsigned>(p.Hkv);
  if (p.tail_tile > 0)  // the last wave's tiles take two blocks each
    return chain_launch(kern, 2 * tiles - static_cast<unsigned>(p.tail_tile), S::THREADS, S::SMEM_ALLOC, stream, 2, *tk,
                        *tv, p);
  return chain_launch(kern, tiles * static_cast<unsigned>(p.splits), S::THREADS, S::SMEM_ALLOC, stream,
                      static_cast<unsigned>(p.cluster), *tk, *tv, p);
}

template <int D>
cudaError_t launch_paged_rows(int tile_rows, const CUtensorMap* tk, const CUtensorMap* tv,
                              const PagedParams& p, cudaStream_t stream) {
  if (tile_rows >= kPrefillRows) return launch_prefill<D>(tk, tv, p, stream);
  switch (tile_rows) {
    case 8:
      return p.page_size == 16 ? launch_paged_shape<PagedShape<D, 1, true>>(tk, tv, p, stream)
                               : launch_paged_shape<PagedShape<D, 1, false>>(tk, tv, p, stream);
    case 16:
      return p.page_size == 16 ? launch_paged_shape<PagedShape<D, 2, true>>(tk, tv, p, stream)
                               : launch_paged_shape<PagedShape<D, 2, false>>(tk, tv, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ea51

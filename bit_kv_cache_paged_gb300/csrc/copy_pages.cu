// Copies of whole pages inside the BF16-only cache (fork of a tail page, compaction).
//
// A page of one layer is contiguous over its KV heads: Hkv x 16 KB of K, as much of V. The work is
// one read and one write of every moved page; memory bounds it. The (source, destination) pairs
// travel as launch parameters, so that no list has to be uploaded or kept alive, and the host has
// checked that no page is written twice or both read and written: copies need no order.
//
// Measured: 32 pages of 8 KV heads in 36 layers (604 MB read and written) 89.7 us, 6730 GB/s, 99% of the
// copy peak; one page of one layer 2.0 us, a launch's own time.
#include <algorithm>
#include <new>
#include <vector>

#include "device_common.cuh"

namespace oscar {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;                                     // 16-byte loads in flight per thread
constexpr int kCopyBytes = kCopyThreads * kCopyUnroll * 16;        // 16 KB of one page per CTA
constexpr int kBf16PageBytes = kPage * kHeadDim * 2;
static_assert(kBf16PageBytes % kCopyBytes == 0, "a CTA copies whole pieces of a page");
// Pairs per launch: 8 KB of parameters, or 512 bytes for the few pairs of a fork, whose launch is
// cheaper on the host.
constexpr int kMaxMoves = 1024, kFewMoves = 64;

template <int N>
struct PageMoves {
  int32_t src[N], dst[N];
};

// blockIdx.x: (pair, piece of the page); y: layer; z: K or V
template <int N>
__global__ void __launch_bounds__(kCopyThreads) k_copy_pages(uint8_t* k, uint8_t* v, size_t layer_stride, int hkv,
                                                            const __grid_constant__ PageMoves<N> M) {
  const int m = blockIdx.x / hkv, piece = blockIdx.x - m * hkv;
  uint8_t* base = (blockIdx.z ? v : k) + (size_t)blockIdx.y * layer_stride;
  const size_t page = (size_t)hkv * kBf16PageBytes, off = (size_t)piece * kCopyBytes + threadIdx.x * 16;
  const uint8_t* s = base + (size_t)M.src[m] * page + off;
  uint8_t* d = base + (size_t)M.dst[m] * page + off;
  uint4 r[kCopyUnroll];
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) r[i] = __ldcs(reinterpret_cast<const uint4*>(s + i * kCopyThreads * 16));
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) *reinterpret_cast<uint4*>(d + i * kCopyThreads * 16) = r[i];
}

template <int N>
cudaError_t launch_copy(uint8_t* k, uint8_t* v, size_t layer_stride, int hkv, int n_layers, const int32_t* src, const int32_t* dst,
                        int32_t m, cudaStream_t st) {
  PageMoves<N> M;
  std::copy(src, src + m, M.src);
  std::copy(dst, dst + m, M.dst);
  const dim3 grid((unsigned)m * (unsigned)hkv, n_layers, 2);
  k_copy_pages<N><<<grid, kCopyThreads, 0, st>>>(k, v, layer_stride, hkv, M);
  return cudaGetLastError();
}

}  // namespace
}  // namespace oscar

using namespace oscar;

extern "C" oscar_status oscar_bf16_copy_pages(int32_t num_kv_heads, int32_t n_layers, size_t layer_stride, void* k_pages,
                                              void* v_pages, int64_t n_pages_total, const int32_t* src,
                                              const int32_t* dst, int32_t n, void* stream) {
  if (num_kv_heads < 1 || n_layers < 1 || n_layers > 65535 || n < 0 || n_pages_total < 1 || !k_pages || !v_pages)
    return OSCAR_EINVAL;
  if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15) != 0) return OSCAR_EINVAL;
  if (n_layers > 1 && (layer_stride % 16 || layer_stride / num_kv_heads / kBf16PageBytes < (uint64_t)n_pages_total))
    return OSCAR_EINVAL;
  if (num_kv_heads > (1 << 20)) return OSCAR_EINVAL;
  if (n == 0) return OSCAR_OK;
  if (!src || !dst) return OSCAR_EINVAL;
  for (int32_t i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= n_pages_total || dst[i] < 0 || dst[i] >= n_pages_total) return OSCAR_EINVAL;
  try {
    std::vector<int32_t> to(dst, dst + n);
    std::sort(to.begin(), to.end());
    for (int32_t i = 1; i < n; ++i)
      if (to[i] == to[i - 1]) return OSCAR_EINVAL;
    for (int32_t i = 0; i < n; ++i)
      if (std::binary_search(to.begin(), to.end(), src[i])) return OSCAR_EINVAL;
  } catch (const std::bad_alloc&) {
    return OSCAR_ENOMEM;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int32_t per = std::min<int64_t>(kMaxMoves, std::max<int64_t>(1, INT32_MAX / num_kv_heads));
  for (int32_t at = 0; at < n; at += per) {
    const int32_t m = std::min(per, n - at);
    uint8_t *k = static_cast<uint8_t*>(k_pages), *v = static_cast<uint8_t*>(v_pages);
    const cudaError_t e = m <= kFewMoves ? launch_copy<kFewMoves>(k, v, layer_stride, num_kv_heads, n_layers, src + at, dst + at, m, st)
                                         : launch_copy<kMaxMoves>(k, v, layer_stride, num_kv_heads, n_layers, src + at, dst + at, m, st);
    if (e != cudaSuccess) return OSCAR_ECUDA;
  }
  return OSCAR_OK;
}

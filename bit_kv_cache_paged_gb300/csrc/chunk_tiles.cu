// The INT2 histories of a step as fp16 tiles, for chunks long enough to use them several times.
//
// Every pair of query tiles of a KV head (256 rows: 64 tokens at 4 query heads) goes over the whole
// history. Dequantising inside the chunk kernel costs each of them the expansion of every block again, on
// the SMs that also run the softmax; made once here, the blocks come in by bulk copies like BF16
// keys. A block costs 9 KB read and 64 KB written here, and 64 KB read (from L2 mostly: the pairs of a
// head follow one another) for each pair.
//
// A tile is stored as the tensor cores read it: two halves of 64 dims, token r of a half 128 bytes at
// r * 128, its 16-byte chunk c at chunk position c ^ (r & 7). A CTA expands a block's K (warps 0-3) and V
// (warps 4-7) into shared memory and sends them out by bulk copies; memory bounds it.
//
// Measured: 29700 tokens of 8 KV heads, group 128 (139 MB read and written) 21 us, 6600 GB/s; the whole call
// of 2048 tokens, replayed from a graph, 705 us, where dequantising in the kernel takes 893.
#include <type_traits>

#include "int2_tiles.cuh"

namespace oscar {
namespace {

constexpr int kTilesThreads = 256;
constexpr int kBlockTokens = 2 * kPage;
constexpr int kTilesSmem = 2 * kInt2TileBytes;
constexpr int kTilesCtas = 3;  // per SM (shared memory)

__device__ __forceinline__ int history_blocks(const StepSeq& st, bool skip_single) {
  const int n = st.L_new - st.L_old;
  return n == 0 || (skip_single && n == 1) ? 0 : (st.F_old - kSink + kBlockTokens - 1) / kBlockTokens;
}

// base[i]: blocks of the sequences before i.
__global__ void __launch_bounds__(kTilesThreads) k_tile_base(DevPool P, int n_seqs, bool skip_single, int32_t* base) {
  __shared__ int32_t scan[kTilesThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t sum = 0;
  for (int i0 = 0; i0 < n_seqs; i0 += kTilesThreads) {
    const int i = i0 + threadIdx.x;
    const int32_t mine = i < n_seqs ? history_blocks(P.step[i], skip_single) : 0;
    int32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int32_t before = sum + inc - mine;
    for (int w = 0; w < kTilesThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      sum += scan[w];
    }
    if (i < n_seqs) base[i] = before;
  }
  if (threadIdx.x == 0) base[n_seqs] = sum;
}

__global__ void __launch_bounds__(kTilesThreads, kTilesCtas)
    k_tiles(DevPool P, int n_seqs, int layer, const int32_t* __restrict__ base, int64_t max_tasks, uint8_t* __restrict__ tiles) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int x = threadIdx.x & 127, kv = threadIdx.x >> 7;
  const int slice = x >> 4, wh = (x >> 3) & 1, uu = (x >> 2) & 1, tq = x & 3;  // V: see chunk.cu
  const int ng = P.ngroups;
  const int64_t tasks = min((int64_t)base[n_seqs] * P.Hkv, max_tasks);
  const bool table = P.lloyd != 0;
  bool sent = false;  // thread 0: a bulk store may still be reading the tiles
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {  // the last sequence that starts at or before the task (empty ones start where the next does)
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)base[mid] * P.Hkv <= task) lo = mid; else hi = mid - 1;
    }
    const StepSeq& st = P.step[lo];
    const int nI = base[lo + 1] - base[lo], rem = (int)(task - (int64_t)base[lo] * P.Hkv), h = rem / nI, k = rem - h * nI;
    const int hist = st.F_old - kSink;
    // this thread's eight packed words, and the (scale, zero) of each of the four times 32 values that they
    // hold; of a token behind the history both are 0, so its values are
    const int half = kv ? slice >> 2 : x >> 6, page = 2 * k + half;
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0}, szw[4] = {0, 0, 0, 0};
    if (page * kPage < hist) {
      int64_t pid = P.page_table[(size_t)st.seq_id * P.maxp + page];
      if (pid < 0 || pid >= P.max_int2_pages) {
        set_err(P.err, OSCAR_DEVERR_PAGE);
        pid = 0;
      }
      const uint8_t* pg = P.int2 + (size_t)layer * P.int2_layer_stride + ((size_t)pid * P.Hkv + h) * P.block_bytes;
      const uint32_t* sz = reinterpret_cast<const uint32_t*>(pg + 2 * kPage * kCodeBytes) + (kv ? kPage * ng : 0);
      if (kv) {
        const uint8_t* src = pg + kPage * kCodeBytes + (slice & 3) * 512 + tq * 16 + 8 * uu + 4 * wh;
#pragma unroll
        for (int g = 0; g < 8; ++g) w[g] = *reinterpret_cast<const uint32_t*>(src + g * 64);
      } else {
        const uint4 c0 = reinterpret_cast<const uint4*>(pg + (x & 63) * kCodeBytes)[0];
        const uint4 c1 = reinterpret_cast<const uint4*>(pg + (x & 63) * kCodeBytes)[1];
        w[0] = c0.x, w[1] = c0.y, w[2] = c0.z, w[3] = c0.w, w[4] = c1.x, w[5] = c1.y, w[6] = c1.z, w[7] = c1.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tau = kv ? (slice & 3) * 16 + 8 * uu + 2 * tq + ((i >> 1) ^ uu) : x & 63;
        if (page * kPage + tau < hist) szw[i] = sz[sz_index(tau, ng == 1 ? 0 : kv ? 2 * wh + (i & 1) : i, ng)];
      }
    }
    const float a = table ? P.cb_a[((size_t)layer * P.Hkv + h) * 2 + kv] : 1.f;
    if (sent) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncthreads();
    const int row0 = kv ? slice * 16 + 8 * uu + 2 * tq : x;
    uint8_t* tile = smem + kv * kInt2TileBytes + (kv ? wh * kTileHalfBytes : 0);
    auto fill = [&](auto tab) {
      constexpr bool T = decltype(tab)::value;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int hi2 = i >> 1, b = i & 1, e = hi2 ^ uu, row = kv ? row0 + e : row0;
        uint8_t* dst = tile + row * 128 + (kv ? 0 : hi2 * kTileHalfBytes);
        const Levels t = levels(szw[i], a, T);
        const uint32_t sel = kv ? (e ? 0x7632u : 0x5410u) : (hi2 ? 0x7654u : 0x3210u);
        uint32_t W[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) W[j] = __byte_perm(w[2 * j], w[2 * j + 1], sel) >> (8 * b);
#pragma unroll
        for (int p = 0; p < 4; ++p)
          *reinterpret_cast<uint4*>(dst + (((4 * b + p) ^ (row & 7)) << 4)) =
              make_uint4(expand(W[0], p, t, T), expand(W[1], p, t, T), expand(W[2], p, t, T), expand(W[3], p, t, T));
      }
    };
    if (table) fill(std::true_type{}); else fill(std::false_type{});
    fence_proxy_async();
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int t = 0; t < 2; ++t)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(tiles + (2 * task + t) * kInt2TileBytes),
                     "r"(smem_u32(smem + t * kInt2TileBytes)), "r"(kInt2TileBytes)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      sent = true;
    }
  }
  if (sent) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

size_t base_bytes(const StepDims& S) { return ((size_t)S.n_seqs + 1 + 63) / 64 * 64 * 4; }

}  // namespace

size_t chunk_tiles_workspace_bytes(const DevPool& P, const StepDims& S, int64_t blocks) {
  return base_bytes(S) + (size_t)blocks * P.Hkv * 2 * kInt2TileBytes;
}

cudaError_t launch_chunk_tiles(const DevPool& P, const StepDims& S, int layer, bool skip_single, int64_t blocks,
                               void* workspace, ChunkTiles* out, cudaStream_t s) {
  int32_t* base = static_cast<int32_t*>(workspace);
  uint8_t* tiles = static_cast<uint8_t*>(workspace) + base_bytes(S);
  out->base = base;
  out->tiles = tiles;
  k_tile_base<<<1, kTilesThreads, 0, s>>>(P, S.n_seqs, skip_single, base);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_tiles, cudaFuncAttributeMaxDynamicSharedMemorySize, kTilesSmem);
  if (e != cudaSuccess) return e;
  const int64_t tasks = blocks * P.Hkv, most = (int64_t)P.num_sms * kTilesCtas;
  k_tiles<<<(unsigned)(tasks < most ? tasks : most), kTilesThreads, kTilesSmem, s>>>(P, S.n_seqs, layer, base, tasks, tiles);
  return cudaGetLastError();
}

}  // namespace oscar

// Attention of a chunk of new tokens over a paged cache: the BF16-only pages (oscar_bf16_chunk), and
// the pool's mixed cache before the step's append (oscar_chunk_attend).
//
//   out[t, h] = sum_s softmax_s(q[t, h] . k[s] / sqrt(128)) v[s],  s over the keys token t sees
//
// One pass with the running maximum and sum of the softmax in base 2. Keys of the INT2 history are
// compared in the rotated basis (k^ = level * s + z, q R_K), their values summed there and un-rotated
// once: R = U H P, so o R^T goes back through the bit reversal, the Walsh-Hadamard transform and U^T.
//
// One warp takes one (token, query head); a lane holds four dims. Each key costs a warp reduction.
#include "device_common.cuh"

namespace oscar {
namespace {

constexpr int kChunkWarps = 8;
constexpr int kChunkPageBytes = kPage * kHeadDim * 2;

struct Bf16Chunk {
  const uint8_t *k, *v;
  const int32_t *page_table, *lengths, *cu;
  int32_t n_seqs, n_tokens, Hq, Hkv, max_pages;
  int64_t n_pages_total, q_stride;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  uint32_t* err;
};

__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The running softmax of one row: maximum (log2 units), sum, unnormalised output.
struct Row {
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const float (&q)[4], const float (&k)[4], const float (&v)[4]) {
    float d = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
    d *= kScoreLog2;
    const float mn = fmaxf(m, d), c = fast_exp2(m - mn), p = fast_exp2(d - mn);
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * c + p * v[e];
    m = mn;
  }
};

__global__ void __launch_bounds__(kChunkWarps * 32) k_bf16_chunk(Bf16Chunk C) {
  const int64_t w = (int64_t)blockIdx.x * kChunkWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / C.Hq), h = (int)(w - (int64_t)t * C.Hq);
  if (t >= C.n_tokens || t < C.cu[0] || t >= C.cu[C.n_seqs]) return;
  int lo = 0, hi = C.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (C.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int kvh = h / (C.Hq / C.Hkv);
  int len = C.lengths[lo];
  if (len > C.max_pages * kPage) {
    set_err(C.err, OSCAR_DEVERR_PAGE);
    len = C.max_pages * kPage;
  }
  const int last = len - (C.cu[lo + 1] - t);  // this token's position
  Row R;
  float q[4], k[4], v[4];
  load4(C.q + (int64_t)t * C.q_stride + (int64_t)h * kHeadDim + 4 * lane, q);
  for (int p = 0; p <= last; ++p) {
    const int64_t pid = C.page_table[(int64_t)lo * C.max_pages + (p >> 6)];
    if (pid < 0 || pid >= C.n_pages_total) {
      set_err(C.err, OSCAR_DEVERR_PAGE);
      continue;
    }
    const size_t off = ((size_t)pid * C.Hkv + kvh) * kChunkPageBytes + bf16_chunk_offset(p & 63, lane >> 1) + (lane & 1) * 8;
    load4(reinterpret_cast<const __nv_bfloat16*>(C.k + off), k);
    load4(reinterpret_cast<const __nv_bfloat16*>(C.v + off), v);
    R.add(q, k, v);
  }
  const float inv = R.l > 0.f ? 1.f / R.l : (R.m == -INFINITY ? 0.f : 1.f / R.l);
#pragma unroll
  for (int e = 0; e < 4; ++e) R.o[e] *= inv;
  store4(C.out + ((int64_t)t * C.Hq + h) * kHeadDim + 4 * lane, R.o);
}

__global__ void __launch_bounds__(kChunkWarps * 32) k_pool_chunk(DevPool P, StepDims S, int layer, const __nv_bfloat16* q_rows,
                                                                 const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                                                                 __nv_bfloat16* out) {
  const int64_t w = (int64_t)blockIdx.x * kChunkWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / P.Hq), h = (int)(w - (int64_t)t * P.Hq);
  if (t >= S.total_new) return;
  int lo = 0, hi = S.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.step[mid].in_offset <= t) lo = mid; else hi = mid - 1;
  }
  const StepSeq st = P.step[lo];
  const int kvh = h / P.hg;
  const size_t lh = (size_t)layer * P.Hkv + kvh;
  Row R;
  float q[4], k[4], v[4];
  load4(q_rows + ((int64_t)t * P.Hq + h) * kHeadDim + 4 * lane, q);
  if (st.F_old > kSink) {
    float x[1][4], y[1][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[0][e] = q[e];
    matvec_u<1>(x, P.Uk + lh * kHeadDim * kHeadDim, y, lane);
    float qr[4] = {y[0][0], y[0][1], y[0][2], y[0][3]};
    fwht128(qr, lane);
    const int ng = P.ngroups;
    const float ak = P.cb_a[lh * 2], av = P.cb_a[lh * 2 + 1];
    auto level = [&](int c, float a) { return P.lloyd ? (c == 0 ? 0.f : c == 3 ? 3.f : c == 1 ? a : 3.f - a) : (float)c; };
    for (int p = kSink; p < st.F_old; ++p) {
      const int pid = P.page_table[(size_t)st.seq_id * P.maxp + ((p - kSink) >> 6)], tau = (p - kSink) & 63;
      if (pid < 0 || pid >= P.max_int2_pages) {
        set_err(P.err, OSCAR_DEVERR_PAGE);
        continue;
      }
      const uint8_t* blk = P.int2 + (size_t)layer * P.int2_layer_stride + ((size_t)pid * P.Hkv + kvh) * P.block_bytes;
      const uint32_t* sz = reinterpret_cast<const uint32_t*>(blk + 2 * kPage * kCodeBytes);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = rot_pos(lane, e);
        const int pb = (j >> 3) & 3;
        const uint8_t kb = blk[tau * kCodeBytes + ((j & 7) >> 1) * 8 + (j >> 6) * 4 + 2 * (j & 1) + ((j >> 5) & 1)];
        const int ts = tau & 15, word = j >> 5;
        const uint8_t vb = blk[kPage * kCodeBytes + (tau >> 4) * 512 + ((j & 7) * 4 + ((ts >> 1) & 3)) * 16 +
                               4 * (2 * (ts >> 3) + (word >> 1)) + 2 * (ts & 1) + (word & 1)];
        const uint32_t ks = sz[sz_index(tau, j / P.G, ng)], vs = sz[kPage * ng + sz_index(tau, j / P.G, ng)];
        k[e] = fmaf(level((kb >> (2 * pb)) & 3, ak), half_lo(ks), half_hi(ks));
        v[e] = fmaf(level((vb >> (2 * pb)) & 3, av), half_lo(vs), half_hi(vs));
      }
      R.add(qr, k, v);
    }
    if (!P.absorbed) {
      fwht128(R.o, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][e] = R.o[e];
      matvec_u<1>(x, P.Utv + lh * kHeadDim * kHeadDim, y, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) R.o[e] = y[0][e];
    } else {  // the rotated basis itself, in its own order
      float y4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // dim 4 lane + e was held by the lane and slot of its bit reversal
        const int i = bitrev7(4 * lane + e);
        float g = 0.f;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const float z = __shfl_sync(0xffffffffu, R.o[f], i >> 2);
          if ((i & 3) == f) g = z;
        }
        y4[e] = g;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) R.o[e] = y4[e];
    }
  }
  const __nv_bfloat16* sk = P.sink_k + (size_t)layer * P.sink_layer_stride + ((size_t)st.sink_page * P.Hkv + kvh) * kPage * kHeadDim;
  const __nv_bfloat16* sv = P.sink_v + (size_t)layer * P.sink_layer_stride + ((size_t)st.sink_page * P.Hkv + kvh) * kPage * kHeadDim;
  for (int p = 0; p < min(kSink, st.L_old); ++p) {
    const int off = (bf16_chunk_offset(p, lane >> 1) + (lane & 1) * 8) / 2;
    load4(sk + off, k);
    load4(sv + off, v);
    R.add(q, k, v);
  }
  const size_t ring = (size_t)layer * P.ring_layer_stride + ((size_t)st.seq_id * P.Hkv + kvh) * kRecent * kHeadDim;
  for (int p = st.F_old; p < st.L_old; ++p) {
    const int off = (bf16_chunk_offset(p & (kRecent - 1), lane >> 1) + (lane & 1) * 8) / 2;
    load4(P.ring_k + ring + off, k);
    load4(P.ring_v + ring + off, v);
    R.add(q, k, v);
  }
  for (int j = 0; j <= t - st.in_offset; ++j) {
    const int64_t off = ((int64_t)(st.in_offset + j) * P.Hkv + kvh) * kHeadDim + 4 * lane;
    load4(k_new + off, k);
    load4(v_new + off, v);
    R.add(q, k, v);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) R.o[e] /= R.l;
  store4(out + ((int64_t)t * P.Hq + h) * kHeadDim + 4 * lane, R.o);
}

}  // namespace

size_t chunk_workspace_bytes(int, int64_t) { return 16; }

cudaError_t launch_chunk_pool(const DevPool& P, const StepDims& S, int layer, const void* q, const void* k_new,
                              const void* v_new, void*, void* out, cudaStream_t s) {
  const int64_t warps = (int64_t)S.total_new * P.Hq;
  k_pool_chunk<<<(unsigned)((warps + kChunkWarps - 1) / kChunkWarps), kChunkWarps * 32, 0, s>>>(
      P, S, layer, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k_new),
      static_cast<const __nv_bfloat16*>(v_new), static_cast<__nv_bfloat16*>(out));
  return cudaGetLastError();
}

}  // namespace oscar

using namespace oscar;

extern "C" {

size_t oscar_bf16_chunk_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t n_seqs, int32_t n_tokens) {
  if (num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads || n_seqs < 1 || n_tokens < 0) return 0;
  const int hg = num_q_heads / num_kv_heads;
  if (hg != 1 && hg != 2 && hg != 4 && hg != 8 && hg != 16) return 0;
  return chunk_workspace_bytes(hg, n_tokens);
}

oscar_status oscar_bf16_chunk(int32_t num_q_heads, int32_t num_kv_heads, int32_t n_seqs, int32_t n_tokens,
                              const void* k_pages, const void* v_pages, int64_t n_pages_total, const int32_t* page_table,
                              int32_t max_pages_per_seq, const int32_t* lengths, const int32_t* cu_tokens, const void* q,
                              int64_t q_token_stride, void* workspace, size_t workspace_bytes, void* out, uint32_t* err,
                              void* stream) {
  const size_t need = oscar_bf16_chunk_workspace_bytes(num_q_heads, num_kv_heads, n_seqs, n_tokens);
  if (!need) return OSCAR_EINVAL;
  if (n_tokens == 0) return OSCAR_OK;
  if (!k_pages || !v_pages || !page_table || !lengths || !cu_tokens || !q || !workspace || !out || !err) return OSCAR_EINVAL;
  if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages) | reinterpret_cast<uintptr_t>(q) |
        reinterpret_cast<uintptr_t>(workspace) | reinterpret_cast<uintptr_t>(out)) & 15) != 0)
    return OSCAR_EINVAL;  // read and written in 16-byte pieces
  if (((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(cu_tokens) |
        reinterpret_cast<uintptr_t>(err)) & 3) != 0)
    return OSCAR_EINVAL;
  if (q_token_stride % 8 || q_token_stride < (int64_t)num_q_heads * kHeadDim) return OSCAR_EINVAL;
  if (workspace_bytes < need || n_pages_total < 1 || n_pages_total > INT32_MAX || max_pages_per_seq < 1 ||
      max_pages_per_seq > INT32_MAX / kPage)
    return OSCAR_EINVAL;
  Bf16Chunk C;
  C.k = static_cast<const uint8_t*>(k_pages);
  C.v = static_cast<const uint8_t*>(v_pages);
  C.page_table = page_table;
  C.lengths = lengths;
  C.cu = cu_tokens;
  C.n_seqs = n_seqs;
  C.n_tokens = n_tokens;
  C.Hq = num_q_heads;
  C.Hkv = num_kv_heads;
  C.max_pages = max_pages_per_seq;
  C.n_pages_total = n_pages_total;
  C.q_stride = q_token_stride;
  C.q = static_cast<const __nv_bfloat16*>(q);
  C.out = static_cast<__nv_bfloat16*>(out);
  C.err = err;
  const int64_t warps = (int64_t)n_tokens * num_q_heads;
  k_bf16_chunk<<<(unsigned)((warps + kChunkWarps - 1) / kChunkWarps), kChunkWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(C);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ECUDA;
}

}  // extern "C"

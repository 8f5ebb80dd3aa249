// Chunk attention of the sequences with one new token, over long INT2 histories.
//
// One token's hg query rows fill 4 or 8 of the 128 rows that a tensor-core tile of chunk.cu has, and each
// 128 keys would still cost it the dequantising of 64 KB: 3.8 thousand cycles where the packed pages
// (9 KB) take 400 to read. The decode kernels take the codes as they lie, so such sequences go
// through them, over the cache as it stands before the step: a small kernel writes that view (step
// description with F_old and L_old for F_new and L_new, INT2 units recounted), then rotate_q, the INT2
// and BF16 decodes and the merge run on it, the merge with the new token itself as one more key.
// Memory bounds it (72 or 96 bytes per history token and KV head).
//
// The BF16 decode needs nothing from the rotation: outside a capture it runs beside it on a branch, joined
// before the merge (64 us a call, 72 without).
//
// Measured at 8 sequences of 32K history, 32 query and 8 KV heads, group 128: 224 us in chunk.cu, here 64 us a
// call, 60 replayed: view 3, rotation 6, BF16 decode 8, INT2 decode 41 (the packed pages alone take 24 us at the
// copy peak; the decode kernel is bound by the unpacking of its codes), merge 11, each with a cold cache.
#include "device_common.cuh"

namespace oscar {
namespace {

constexpr int kViewThreads = 256;

// The view of the single-token sequences, and their q rows gathered (q_out null: they lie in order
// already). Every block scans the batch, block 0 writes the view, all share the rows.
__global__ void __launch_bounds__(kViewThreads) k_view(DevPool P, StepDims S, StepDims S1, StepDims* dims,
                                                       StepSeq* steps, const uint4* __restrict__ q, uint4* __restrict__ q_out) {
  __shared__ int64_t scan[kViewThreads / 32][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t n = 0, units = 0;  // of the sequences before this round
  for (int i0 = 0; i0 < S.n_seqs; i0 += kViewThreads) {
    const int i = i0 + threadIdx.x;
    StepSeq st{};
    if (i < S.n_seqs) st = P.step[i];
    const bool mine = st.L_new - st.L_old == 1;
    const int pages = mine && st.F_old > kSink ? (st.F_old - kSink + kPage - 1) / kPage : 0;
    int64_t a = mine ? 1 : 0, u = (int64_t)pages * P.Hkv;
    const int64_t u0 = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) {
        a += x;
        u += y;
      }
    }
    __syncthreads();
    if (lane == 31) {
      scan[warp][0] = a;
      scan[warp][1] = u;
    }
    __syncthreads();
    int64_t at = n + a - 1, before = units + u - u0;
    for (int w = 0; w < kViewThreads / 32; ++w) {
      if (w < warp) {
        at += scan[w][0];
        before += scan[w][1];
      }
      n += scan[w][0];
      units += scan[w][1];
    }
    if (mine && at < S1.n_seqs) {
      if (blockIdx.x == 0) {
        StepSeq v = st;
        v.L_new = st.L_old;
        v.F_new = st.F_old;
        v.n_pages = pages;
        v.unit_offset = (int32_t)before;
        steps[at] = v;
      }
      if (q_out) {
        // rows of 256 bytes, by the blocks in turn
        for (int c = blockIdx.x; c < P.Hq * (kHeadDim / 8); c += gridDim.x)
          q_out[at * P.Hq * (kHeadDim / 8) + c] = q[(int64_t)st.in_offset * P.Hq * (kHeadDim / 8) + c];
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    StepDims d = S1;
    d.total_units = (int32_t)units;
    d.nw = int2_workers(units, S1.n_pairs, S1.nw_max);
    *dims = d;
  }
}

struct SingleBuffers {
  size_t dims, steps, q, q_rot, partials, total;
};
SingleBuffers single_buffers(const DevPool& P, const StepDims& S1) {
  SingleBuffers b{};
  auto take = [&](size_t bytes) {
    const size_t at = b.total;
    b.total += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t rows = (size_t)S1.n_seqs * P.Hq * kHeadDim;
  b.dims = take(sizeof(StepDims));
  b.steps = take((size_t)S1.n_seqs * sizeof(StepSeq));
  b.q = take(rows * 2);
  b.q_rot = take(rows * 4);
  b.partials = take(partial_slots(S1) * (size_t)slot_floats(P.hg) * 4);
  return b;
}

}  // namespace

size_t chunk_single_workspace_bytes(const DevPool& P, const StepDims& S1) { return single_buffers(P, S1).total; }

cudaError_t launch_chunk_single(const DevPool& P, const StepDims& S, const StepDims& S1, int layer,
                                const void* q, const void* k_new, const void* v_new, void* workspace, void* out,
                                const ChunkBranch& branch, cudaStream_t s, int* launches) {
  const SingleBuffers b = single_buffers(P, S1);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  StepDims* dims = reinterpret_cast<StepDims*>(ws + b.dims);
  StepSeq* steps = reinterpret_cast<StepSeq*>(ws + b.steps);
  float* q_rot = reinterpret_cast<float*>(ws + b.q_rot);
  float* pbf16 = reinterpret_cast<float*>(ws + b.partials);
  float* pint2 = pbf16 + int2_slot_offset(S1) * slot_floats(P.hg);
  const bool gather = S.total_new != S1.n_seqs;
  const void* q1 = gather ? ws + b.q : q;
  k_view<<<gather ? 16 : 1, kViewThreads, 0, s>>>(P, S, S1, dims, steps, static_cast<const uint4*>(q),
                                                 gather ? reinterpret_cast<uint4*>(ws + b.q) : nullptr);
  cudaError_t e = cudaGetLastError();
  DevPool V = P;  // the pool before the step, as far as the decode kernels look at it
  V.dims = dims;
  V.step = steps;
  *launches = 1;
  auto then = [&](cudaError_t r) {
    e = r;
    ++*launches;
  };
  const bool beside = e == cudaSuccess && branch.side;
  cudaStream_t bs = beside ? branch.side : s;
  if (beside) {
    e = cudaEventRecord(branch.fork, s);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(bs, branch.fork, 0);
    if (e != cudaSuccess) return e;
  }
  if (e == cudaSuccess) then(launch_decode_bf16(V, S1, layer, q1, pbf16, bs));
  if (beside) {
    const cudaError_t r = cudaEventRecord(branch.join, bs);
    if (e == cudaSuccess) e = r;
  }
  if (e == cudaSuccess) then(launch_rotate_q(V, S1, layer, q1, q_rot, s));
  if (e == cudaSuccess) then(launch_decode_int2(V, S1, layer, q_rot, pint2, s));
  if (beside) {
    const cudaError_t r = cudaStreamWaitEvent(s, branch.join, 0);  // the branch joins even after an error
    if (e == cudaSuccess) e = r;
  }
  if (e == cudaSuccess) then(launch_merge_new(V, S1, layer, pint2, pbf16, q1, k_new, v_new, out, s));
  return e;
}

}  // namespace oscar

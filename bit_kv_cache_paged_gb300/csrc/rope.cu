// Rotary positions of query and key rows, before they enter a cache.
//
// Pair j of a token at position p turns by p * w_j: (x_a, x_b) -> A (x_a cos - x_b sin, x_b cos +
// x_a sin). In fp32 the product p * w_j of a far position has lost the fraction of a turn that
// matters (at p = 10^6 an ulp is 0.06 rad). Here w_j / 2 pi is a 64-bit fixed-point fraction of a
// turn, so the product modulo one turn is an integer multiplication that wraps: exact to 2^-53 of
// w_j, whatever p. Its top 32 bits go through sincospif.
//
// The work is one read and one write of every row; memory bounds it. A CTA takes one token: its
// first rot_dim/2 threads make the token's cos and sin once for all heads (shared memory), each
// thread having the 16-byte loads of up to four rows in flight meanwhile.
//
// Measured: 8192 tokens of 64 + 8 heads 53.0 us, 5700 GB/s, 84% of the copy peak (55.7 with two rows in
// flight); 4097 tokens of 16 + 4 heads 8.6 us; 32 tokens of 32 + 8 heads 2.6 us, a launch's own time.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "device_common.cuh"

namespace oscar {
namespace {

constexpr int kRopeThreads = 256;  // at most; kRopeRows head rows of 8 threads each are in flight per thread
constexpr int kRopeRows = 4;
constexpr double kTwoPi = 6.283185307179586476925286766559;

struct RopeRows {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  int64_t xs, ys;  // token strides, elements
  int32_t heads;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight threads per head row, two 16-byte chunks each: thread c of a row of halves takes chunks c
// and c + r/16 (the two sides of 8 pairs) while c < r/16, the threads after that two chunks of the
// copied dims; interleaved pairs lie inside a chunk, thread c takes chunks 2c and 2c + 1.
template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ oscar_rope R, RopeRows Q, RopeRows K,
                                                       const int32_t* __restrict__ positions) {
  __shared__ float2 cs[64];
  const int64_t tok = blockIdx.x;
  const int items = (Q.heads + K.heads) * 8, half = R.rot_dim >> 1;
  const __nv_bfloat16* xq = Q.x + tok * Q.xs;
  const __nv_bfloat16* xk = K.x + tok * K.xs;
  __nv_bfloat16* yq = Q.y + tok * Q.ys;
  __nv_bfloat16* yk = K.y + tok * K.ys;
  const int c = threadIdx.x & 7;
  const int hc = half >> 3;  // chunks of one side
  int c0, c1;
  bool turn0, turn1;
  if (INTER) {
    c0 = 2 * c;
    c1 = c0 + 1;
    turn0 = c0 * 8 < R.rot_dim;
    turn1 = c1 * 8 < R.rot_dim;
  } else {
    turn0 = turn1 = c < hc;
    c0 = turn0 ? c : 2 * hc + 2 * (c - hc);
    c1 = turn0 ? c + hc : c0 + 1;
  }
  auto src = [&](int i) {
    const int h = i >> 3;
    return h < Q.heads ? xq + h * kHeadDim : xk + (h - Q.heads) * kHeadDim;
  };
  const int step = blockDim.x;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < items; i0 += kRopeRows * step) {
    uint4 a[kRopeRows], b[kRopeRows];
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      if (i0 + r * step < items) {
        const uint4* p = reinterpret_cast<const uint4*>(src(i0 + r * step));
        a[r] = p[c0];
        b[r] = p[c1];
      }
    }
    if (i0 == threadIdx.x) {  // the first time round
      if (threadIdx.x < half) {
        const uint64_t turn = (uint64_t)(int64_t)positions[tok] * R.turns[threadIdx.x];
        float s, co;
        sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077392578125e-10f, &s, &co);  // 2^-31 of half a turn
        cs[threadIdx.x] = make_float2(R.amplitude * co, R.amplitude * s);
      }
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      const int i = i0 + r * step;
      if (i >= items) break;
      const int h = i >> 3;
      __nv_bfloat16* y = h < Q.heads ? yq + h * kHeadDim : yk + (h - Q.heads) * kHeadDim;
      float fa[8], fb[8];
      unpack8(a[r], fa);
      unpack8(b[r], fb);
      if (INTER) {
        auto spin = [&](float (&f)[8], int chunk) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t = cs[chunk * 4 + e];
            const float u = f[2 * e], v = f[2 * e + 1];
            f[2 * e] = u * t.x - v * t.y;
            f[2 * e + 1] = v * t.x + u * t.y;
          }
        };
        if (turn0) {
          spin(fa, c0);
          a[r] = pack8(fa);
        }
        if (turn1) {
          spin(fb, c1);
          b[r] = pack8(fb);
        }
      } else if (turn0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 t = cs[c0 * 8 + e];
          const float u = fa[e], v = fb[e];
          fa[e] = u * t.x - v * t.y;
          fb[e] = v * t.x + u * t.y;
        }
        a[r] = pack8(fa);
        b[r] = pack8(fb);
      }
      uint4* o = reinterpret_cast<uint4*>(y);
      o[c0] = a[r];
      o[c1] = b[r];
    }
  }
}

// Whether rows of w bytes at a (every sa bytes) and at b (every sb) share bytes, n rows each; false
// only when they surely do not.
bool rows_overlap(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t w, int64_t n) {
  if (a + (n - 1) * sa + w <= b || b + (n - 1) * sb + w <= a) return false;
  if (sa != sb) return true;
  const int64_t d = (int64_t)((b > a ? b - a : a - b) % (uint64_t)sa);
  return !(d >= w && sa - d >= w);
}

bool rows_ok(const void* x, int64_t xs, const void* y, int64_t ys, int32_t heads, int64_t n) {
  if (heads == 0) return !x && !y;
  if (heads < 0 || heads > (1 << 20) || !x || !y) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const int64_t w = (int64_t)heads * kHeadDim;
  if (((a | b) & 15) || xs % 8 || ys % 8 || xs < w || ys < w || xs > (1ll << 40) || ys > (1ll << 40)) return false;
  if (a == b && xs == ys) return true;  // in place
  return !rows_overlap(a, 2 * xs, b, 2 * ys, 2 * w, n);
}

}  // namespace
}  // namespace oscar

using namespace oscar;

extern "C" {

oscar_status oscar_rope_init(const oscar_rope_config* c, oscar_rope* out) {
  if (!c || !out) return OSCAR_EINVAL;
  if (c->rot_dim < 16 || c->rot_dim > kHeadDim || c->rot_dim % 16) return OSCAR_EINVAL;
  if ((c->interleaved != 0 && c->interleaved != 1) || c->scaling < OSCAR_ROPE_NONE || c->scaling > OSCAR_ROPE_RAMP)
    return OSCAR_EINVAL;
  if (!(c->base > 1.0) || !std::isfinite(c->base) || !(c->factor >= 1.0) || !std::isfinite(c->factor)) return OSCAR_EINVAL;
  if (c->scaling == OSCAR_ROPE_NONE && c->factor != 1.0) return OSCAR_EINVAL;
  if (!(c->amplitude >= 0.0) || !std::isfinite((float)c->amplitude)) return OSCAR_EINVAL;
  const int r = c->rot_dim;
  double base = c->base, lo = 0.0, hi = 0.0;
  if (c->scaling == OSCAR_ROPE_BASE) base *= std::pow(c->factor, (double)r / (r - 2));
  if (!std::isfinite(base)) return OSCAR_EINVAL;
  if (c->scaling == OSCAR_ROPE_RAMP) {
    if (c->original_len < 1 || !(c->beta_slow > 0.0) || !(c->beta_fast >= c->beta_slow) || !std::isfinite(c->beta_fast))
      return OSCAR_EINVAL;
    // the pair index that turns t times within original_len positions
    auto at = [&](double t) { return r * std::log(c->original_len / (t * kTwoPi)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(at(c->beta_fast)), 0.0);
    hi = std::min(std::ceil(at(c->beta_slow)), (double)(r - 1));
  }
  std::memset(out, 0, sizeof(*out));
  out->rot_dim = r;
  out->interleaved = c->interleaved;
  out->amplitude = (float)(c->amplitude > 0.0 ? c->amplitude
                           : c->scaling == OSCAR_ROPE_RAMP ? 0.1 * std::log(c->factor) + 1.0 : 1.0);
  for (int j = 0; j < r / 2; ++j) {
    double w = std::pow(base, -2.0 * j / r);
    if (c->scaling == OSCAR_ROPE_LINEAR) w /= c->factor;
    if (c->scaling == OSCAR_ROPE_RAMP) {
      const double t = std::min(1.0, std::max(0.0, (j - lo) / std::max(hi - lo, 0.001)));
      w = w / c->factor * t + w * (1.0 - t);
    }
    out->turns[j] = (uint64_t)std::ldexp(w / kTwoPi, 64);  // w <= 1: below 2^62
  }
  return OSCAR_OK;
}

oscar_status oscar_rope_apply(const oscar_rope* rope, int32_t n, const int32_t* positions, int32_t num_q_heads,
                              const void* q, int64_t qs, void* q_out, int64_t qos, int32_t num_k_heads, const void* k,
                              int64_t ks, void* k_out, int64_t kos, void* stream) {
  if (!rope || n < 0 || rope->rot_dim < 16 || rope->rot_dim > kHeadDim || rope->rot_dim % 16 ||
      (rope->interleaved != 0 && rope->interleaved != 1))
    return OSCAR_EINVAL;
  if (n == 0) return OSCAR_OK;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3) || num_q_heads < 0 || num_k_heads < 0 ||
      (int64_t)num_q_heads + num_k_heads < 1)
    return OSCAR_EINVAL;
  if (!rows_ok(q, qs, q_out, qos, num_q_heads, n) || !rows_ok(k, ks, k_out, kos, num_k_heads, n)) return OSCAR_EINVAL;
  const RopeRows Q{static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(q_out), qs, qos, num_q_heads};
  const RopeRows K{static_cast<const __nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(k_out), ks, kos, num_k_heads};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // threads that divide the token's rows evenly, at least one per pair
  const int64_t items = 8 * ((int64_t)num_q_heads + num_k_heads), rounds = (items + kRopeThreads - 1) / kRopeThreads;
  const int threads = (int)std::max<int64_t>(64, ((items + rounds - 1) / rounds + 31) / 32 * 32);
  if (rope->interleaved)
    k_rope<true><<<n, threads, 0, st>>>(*rope, Q, K, positions);
  else
    k_rope<false><<<n, threads, 0, st>>>(*rope, Q, K, positions);
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ECUDA;
  return OSCAR_OK;
}

}  // extern "C"

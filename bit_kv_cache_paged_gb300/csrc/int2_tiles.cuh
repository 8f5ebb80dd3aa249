// Expansion of packed INT2 codes to fp16 values, for the tensor-core tiles of the chunk attention
// (chunk.cu, chunk_tiles.cu).
#pragma once

#include "device_common.cuh"

namespace oscar {

constexpr int kTileHalfBytes = 128 * 128;             // 64 dims of 128 tokens
constexpr int kInt2TileBytes = 2 * kTileHalfBytes;    // 128 tokens x 128 dims in fp16

// What turns a group's codes into fp16 values: scale and zero, or with a Lloyd-Max codebook the four
// values as two words that a byte selector picks from (fp32 products, one rounding).
struct Levels {
  uint32_t a, b;
};
__device__ __forceinline__ Levels levels(uint32_t sz, float l1, bool table) {
  Levels r;
  if (table) {
    const float s = half_lo(sz), z = half_hi(sz);
    r.a = pack_half2(z, fmaf(l1, s, z));
    r.b = pack_half2(fmaf(3.f - l1, s, z), fmaf(3.f, s, z));
  } else {
    r.a = __byte_perm(sz, sz, 0x1010);
    r.b = __byte_perm(sz, sz, 0x3232);
  }
  return r;
}
// Slot p (bits 2p, 2p + 1 of either 16-bit half) of x as an f16x2 pair of values. Uniform levels: the
// code bits under the exponent of 2^(10 - 2p) are 2^(10 - 2p) + code, exactly; one subtraction and
// one fused multiply-add (one rounding) make code * s + z.
__device__ __forceinline__ uint32_t expand(uint32_t x, int p, const Levels& t, bool table) {
  if (table) {
    const uint32_t sel = ((x >> (2 * p)) & 0x00030003u) * 0x22u + 0x00100010u;  // nibbles 2c, 2c + 1 per code
    return __byte_perm(t.a, t.b, __byte_perm(sel, 0, 0x4420));
  }
  const uint32_t base = (0x6400u - 0x800u * p) * 0x10001u;
  const uint32_t h = (x & (0x00030003u << (2 * p))) | base;
  const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&base));
  const __half2 v = __hfma2(c, *reinterpret_cast<const __half2*>(&t.a), *reinterpret_cast<const __half2*>(&t.b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace oscar

// Wrappers of the tcgen05 and tensor-copy instructions shared by the tensor-core kernels, and the driver's
// tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "device_common.cuh"

namespace oscar {

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One box of a 3-D tensor map into shared memory; completion counted on the mbarrier.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's tensor-memory lane, issued without waiting, and
// the wait that makes an issued load's registers readable (the registers pass through the wait, so
// no use of them can move above it).
__device__ __forceinline__ void tc_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_ld_wait_pass(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_ld_wait1(uint32_t (&a)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tc_ld_wait_pass(a);
}
// cuTensorMapEncodeTiled from the driver (looked up once; null when unavailable)
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}


// 16 columns, issued, and the wait for every load issued so far, which these registers pass through.
__device__ __forceinline__ void tc_ld16_issue(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tc_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// The way back: N consecutive 32-bit columns of this thread's lane, and the wait for such stores. A store
// issued while another is in flight costs some 250 cycles where one alone costs 30 to 50 (64 columns
// in one store 52, in two 513): one store, or a wait behind each.
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
__device__ __forceinline__ void tc_st64(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x64.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(r[32]), "r"(r[33]), "r"(r[34]), "r"(r[35]), "r"(r[36]), "r"(r[37]), "r"(r[38]), "r"(r[39]), "r"(r[40]), "r"(r[41]), "r"(r[42]), "r"(r[43]), "r"(r[44]), "r"(r[45]), "r"(r[46]), "r"(r[47]), "r"(r[48]), "r"(r[49]), "r"(r[50]), "r"(r[51]), "r"(r[52]), "r"(r[53]), "r"(r[54]), "r"(r[55]), "r"(r[56]), "r"(r[57]), "r"(r[58]), "r"(r[59]), "r"(r[60]), "r"(r[61]), "r"(r[62]), "r"(r[63])
               : "memory");
}
__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One box of a 2-D tensor map into shared memory.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The upper word of the shared-memory descriptors used here: 128-byte swizzle, descriptor version of
// the sm_100 family, 1024 bytes from 8 rows to the next 8. The lower word holds the address and the
// leading offset in 16-byte units.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// One lane of a converged warp (non-zero there).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}

// D[tmem] (+)= A . B^T of 128 x 128 x 128, kind::f16, as eight steps of 16: A and B tiles in shared
// memory K-major, their 128 columns two halves of 16 KB (a, b: lower descriptor words); or A in tensor
// memory (two 16-bit values a column) and B's tile with its N axis contiguous. The whole warp comes
// here, so that addresses stay in uniform registers, and the elected lane issues: with a branch
// around each product, issuing one took twice as long as computing it.
__device__ __forceinline__ void tc_gemm_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 x;\n .reg .b64 a, b;\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n setp.ne.b32 e, %6, 0;\n"
      " add.u32 x, %1, 0;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 0;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n"
      " add.u32 x, %1, 2;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 2;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 4;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 4;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 6;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 6;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1024;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 1024;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1026;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 1026;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1028;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 1028;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1030;\n mov.b64 a, {x, %4};\n add.u32 x, %2, 1030;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"((uint32_t)accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tc_gemm_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 x, y;\n .reg .b64 b;\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n setp.ne.b32 e, %6, 0;\n"
      " add.u32 y, %1, 0;\n add.u32 x, %2, 0;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, p;\n"
      " add.u32 y, %1, 8;\n add.u32 x, %2, 128;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      " add.u32 y, %1, 16;\n add.u32 x, %2, 256;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      " add.u32 y, %1, 24;\n add.u32 x, %2, 384;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      " add.u32 y, %1, 32;\n add.u32 x, %2, 512;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      " add.u32 y, %1, 40;\n add.u32 x, %2, 640;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      " add.u32 y, %1, 48;\n add.u32 x, %2, 768;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      " add.u32 y, %1, 56;\n add.u32 x, %2, 896;\n mov.b64 b, {x, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"((uint32_t)accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tc_commit_elected(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

}  // namespace oscar

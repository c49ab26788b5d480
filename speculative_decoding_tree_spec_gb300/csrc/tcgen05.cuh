// tcgen05.cuh -- inline PTX of the fifth-generation tensor cores used by the attention
// kernel: matrix descriptors, MMAs with A in shared or tensor memory, tensor-memory loads
// and stores.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace svk {

// Shared-memory matrix descriptor of a tile with the 128-byte swizzle: rows of 128 bytes in
// 1024-byte groups of 8, descriptor version 1; `lead` is the distance of the next 64 elements
// of the rows' direction (used where that direction is M or N), in bytes.
__device__ __forceinline__ uint64_t sw128_tile(uint32_t smem_addr, uint32_t lead) {
  uint64_t d = (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lead >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
// Instruction descriptor, kind::f16: bf16 A and B, fp32 accumulator, M = 128, N; A (and B unless
// `b_mn`) K-major.
constexpr uint32_t bf16_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void tc05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tc05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tc05_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tc05_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// One lane of a converged warp.  The MMA issuer's loop runs in the whole warp, so that its
// descriptors are warp-uniform values, and only the instructions themselves stand under this.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kFull, x, 0); }
__device__ __forceinline__ void tc05_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tc05_alloc(uint32_t* smem_addr, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                   smem_u32(smem_addr)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tc05_dealloc(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols)
               : "memory");
}

#define SVK_R4(m, i) m(i), m(i + 1), m(i + 2), m(i + 3)
#define SVK_R16(m, i) SVK_R4(m, i), SVK_R4(m, i + 4), SVK_R4(m, i + 8), SVK_R4(m, i + 12)
#define SVK_R32(m) SVK_R16(m, 0), SVK_R16(m, 16)
#define SVK_OUT(i) "=r"(r[i])
#define SVK_TIE(i) "+r"(r[i])
#define SVK_IN(i) "r"(r[i])
#define SVK_LIST16 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}"
#define SVK_LIST32                                                                             \
  "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24," \
  "%25,%26,%27,%28,%29,%30,%31}"

// 32 consecutive 32-bit columns of this thread's tensor-memory lane.  The loads are issued
// here; tc05_wait_ld and then tc05_landed(r) stand before the first use of r.
__device__ __forceinline__ void tc05_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " SVK_LIST32 ", [%32];\n"
               : SVK_R32(SVK_OUT)
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc05_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 " SVK_LIST16 ", [%16];\n"
               : SVK_R16(SVK_OUT, 0)
               : "r"(taddr)
               : "memory");
}
// 32 columns of 16 lanes (from the address's lane on), as four 16 x 8 pieces: r[4 g], r[4 g + 1] columns 8 g + 2 (t % 4)
// and the next one of lane t / 4, t the thread; r[4 g + 2], r[4 g + 3] of lane t / 4 + 8.
__device__ __forceinline__ void tc05_ld_pieces(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 " SVK_LIST16 ", [%16];\n"
               : SVK_R16(SVK_OUT, 0)
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc05_landed16(uint32_t* r) {
  asm volatile("" : SVK_R16(SVK_TIE, 0));
}
__device__ __forceinline__ void tc05_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], " SVK_LIST16 ";\n" ::SVK_R16(SVK_IN, 0),
               "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc05_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
// Ties the registers to this point: no use of them moves above the wait.
__device__ __forceinline__ void tc05_landed(uint32_t* r) {
  asm volatile("" : SVK_R32(SVK_TIE));
}
__device__ __forceinline__ void tc05_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " SVK_LIST32 ";\n" ::SVK_R32(SVK_IN),
               "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc05_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y,
                                            int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

}  // namespace svk

// PTX of the 16-bit products: tcgen05 kind::f16 with operands of either major order, and
// rank-3 TMA tile loads.  Complements sm100_ptx.cuh.
#pragma once

#include "sm100_ptx.cuh"

namespace moe {
namespace ptx {

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Instruction descriptor of kind::f16: fp16 or bf16 A and B, fp32 D; a_mn / b_mn: the operand
// is MN-major (its rows in shared memory run along M or N) instead of K-major.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4)                                        // D format: f32
         | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10)  // A, B format
         | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16)
         | ((uint32_t)(N >> 3) << 17)                     // N / 8
         | ((uint32_t)(M >> 4) << 24);                    // M / 16
}

// SMEM descriptor of an MN-major operand laid out by 128-byte-swizzled loads of
// [64 k][64 mn] boxes: rows of 128 bytes along MN, 8-k groups 1024 bytes apart, the next 64
// values of MN one box (8192 bytes) on.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(const void* tile) {
  const uint64_t addr = smem_u32(tile);
  uint64_t d = (addr & 0x3FFFFull) >> 4;   // start address (16-byte units)
  d |= (uint64_t)(8192 >> 4) << 16;        // leading byte offset: next 64 values of MN
  d |= (uint64_t)(1024 >> 4) << 32;        // stride byte offset: next 8 values of K
  d |= 1ull << 46;                          // descriptor version (sm_100)
  d |= 2ull << 61;                          // 128-byte swizzle
  return d;
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T over one 16-wide K block, kind::f16, one CTA.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// As mma_f16_ss, over a CTA pair (M = 256: 128 rows of A and half of B's rows in each CTA).
__device__ __forceinline__ void mma_f16_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Rank-3 tile load into this CTA's shared memory completing on the pair leader's barrier
// (`bar_cluster_addr`: the barrier's cluster-window address).  No multicast.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                                 uint32_t bar_cluster_addr) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Arrive on a barrier of another CTA of the cluster without waiting for this thread's earlier
// stores (mbar_arrive_cluster releases them: a round trip to L2 while stores are in flight).
// For handing back TMEM whose reads tcgen05.wait::ld has completed.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr) : "memory");
}

// 16 TMEM lanes x 32 columns as matrix fragments: register 4 g + r of lane l holds lane
// l / 4 + 8 (r / 2) (of the 16 from the address on), column 8 g + 2 (l % 4) + r % 2.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed on the way: lane 8 m + k gives the address of
// the 16 bytes that column k of matrix m occupies; register m of lane l holds row l / 4, columns
// 2 (l % 4) and + 1 of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Copy from this CTA's shared memory to a cluster CTA's (cluster-window addresses of the
// destination and of the barrier there that counts the bytes); size a multiple of 16.
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

}  // namespace ptx
}  // namespace moe

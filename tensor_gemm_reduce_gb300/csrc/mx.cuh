// mx.cuh -- products of e4m3 operands whose scales the tensor cores apply (tcgen05
// kind::mxf8f6f4), written from the public PTX ISA.
#pragma once
#include "ops_common.cuh"

namespace grs {

// D (+)= A B with the scales of one step, bytes of the words in TMEM that idesc_step
// names.  kPair = 2: a CTA pair shares the MMA; the scales of A's rows lie in the TMEM of
// the CTA whose rows they are, those of B's columns in both.
template <int kPair>
__device__ __forceinline__ void mma_scaled(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
  if constexpr (kPair == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes from shared memory to four columns of TMEM, once for each of the
// four groups of 32 lanes (of both CTAs of a pair, each from its own shared memory).
template <int kPair>
__device__ __forceinline__ void copy_scales(uint32_t d_tmem, uint64_t desc) {
  if constexpr (kPair == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(d_tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(d_tmem), "l"(desc) : "memory");
}
// Its source, 512 bytes: unswizzled, groups of 8 rows follow one another.  Row l holds the
// words of rows (or columns) l, l + 32, l + 64 and l + 96 of the operand.
__device__ __forceinline__ uint64_t scales_desc(uint32_t saddr) {
  return desc_join(((saddr & 0x3FFFFu) >> 4) | (128u >> 4) << 16, (128u >> 4) | 1u << 14);
}

// Instruction descriptor of kind::mxf8f6f4: fp32 accumulator, e4m3 operands, ue8m0 scales.
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, int a_mn_major, int b_mn_major) {
  return ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27);
}
__device__ __forceinline__ uint32_t idesc_step(uint32_t idesc, uint32_t id) { return idesc | (id << 4) | (id << 29); }

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, e4m3 operands, no scales.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn_major, int b_mn_major) {
  return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// One lane of a converged warp.  Loops that issue MMAs run in whole warps, so that
// their descriptors stay uniform, and this lane alone issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

// 32 lanes x 16 consecutive columns, complete on return.
__device__ __forceinline__ void tmem_ld_16_columns(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ uint32_t load_u8(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_u32(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

}  // namespace grs

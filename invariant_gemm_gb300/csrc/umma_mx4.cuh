// tcgen05 helpers for block-scaled 4-bit operands (kind::mxf4: E2M1 values,
// one E8M0 scale per 32 along K, FP32 accumulation).
//
// Operands: K-major tiles of 128-byte rows (256 values) with 128-byte swizzle,
// as in umma.cuh; one MMA takes 64 values of K, so a K step moves the start
// address by 32 bytes. Scale factors are read from tensor memory. For 128 rows
// x 128 k they fill 4 columns: lane l of column c holds the four bytes of row
// 32 c + l, in all four 32-lane partitions. The MMA of K step s (of the two in
// those 128 k) takes bytes 2 s, 2 s + 1, chosen by the scale factor ID 2 s of
// the instruction descriptor. 256 rows take 8 columns.
#pragma once

#include "umma.cuh"

namespace ig {

#ifdef __CUDACC__

// kind::mxf4 descriptor, K = 64: E2M1 A and B, E8M0 scales, m x n; `sf` is the
// scale factor ID (0 or 2) of both operands.
__host__ __device__ constexpr uint32_t umma_idesc_mx4(int m, int n) {
  return (1u << 7)                       // A format: E2M1
         | (1u << 10)                    // B format: E2M1
         | ((uint32_t)(n >> 3) << 17)    // N / 8
         | (1u << 23)                    // scale format: E8M0
         | ((uint32_t)(m >> 7) << 27);   // M / 128
}
__host__ __device__ constexpr uint32_t umma_idesc_sf(uint32_t idesc, uint32_t sf) {
  return idesc | (sf << 4) | (sf << 29);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A value that is the same in all lanes, known as such to the compiler. Copies
// and MMAs take their operands from uniform registers: with a warp number,
// loop counters and addresses that it can see to be uniform they are there
// already, else each instruction is preceded by moves (75 cycles to an MMA
// issued by `if (lane == 0)`).
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}

// mbar_wait_bounded by a whole warp, with one answer for all its lanes (what
// follows a wait here are warp-wide tcgen05 instructions).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status,
                                          long long budget = 1ll << 31) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, status, budget));
}

// Descriptor of a 512-byte scale tile in shared memory: 32 rows of 16 bytes,
// no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sf_tile_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// Scale tile, shared memory -> 4 columns of tensor memory, the 32 lanes
// repeated in the four partitions. Ordered before later MMAs of the thread.
__device__ __forceinline__ void sf_tile_to_tmem(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// One block-scaled MMA (issued by a single thread): D = A B^T (+ D).
__device__ __forceinline__ void umma_mx4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb),
        "r"((uint32_t)accumulate)
      : "memory");
}

#endif  // __CUDACC__

}  // namespace ig

// What the attention kernels of few rows share, over caches of 16 and of 8 bits.
#pragma once

#include "tq_attention_line.cuh"

namespace tq {
namespace {

constexpr int kRowsThreads = 160;  // four consumer warps, one producer warp
constexpr int kTileCost = 64;      // start and end of a tile, as one unit
constexpr int kMinPart = 128;      // no CTA gets less than a tile of one unit costs

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Byte offset of 16-byte chunk `chunk` of row `row` in a tile of `rows` rows kept as 64-element blocks of 128-byte rows
// in the 128-byte swizzle (as TMA writes it).
__device__ __forceinline__ uint32_t sw_off(int rows, int row, int chunk) {
  return (uint32_t)(((chunk >> 3) * rows + row) * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// Gives a ring entry of V back to TMA. A load that was issued may still be under way when an arrival behind it is seen and TMA
// writes the next tile there, and nothing keeps a product before an arrival that does not need it. So the arrival's address takes
// bits of all products, `used`, times a 0 that the compiler does not know (a batch is not negative). K's entry is given
// back behind the barrier that the weights made of it are stored before. With the arrivals right behind the loads' issue 16 requests
// of 4096 to 8192 tokens, 32 heads on 8 of 128, took 62.4 us, as they do so; over 8 bits tiles of 32 rows took 0.5 to 1.4 % less.
__device__ __forceinline__ void give_back(uint64_t* bar, uint32_t used, int batch) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar) + (used & (uint32_t)(batch >> 31))) : "memory");
}
template <int N>
__device__ __forceinline__ uint32_t bits_of(const float (&c)[N][4]) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) r |= __float_as_uint(c[i][0]);
  return r;
}

// Barrier over the four consumer warps; true for all where the predicate is true for one.
__device__ __forceinline__ bool consumers_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

}  // namespace
}  // namespace tq

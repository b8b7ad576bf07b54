// The 4-bit operand format shared by the group-scaled layers (w4_*.cu) and the key/value cache
// (kv4_*.cu), and the device helpers that read it.
//
// Codes are held in the order in which the warp-level matrix instruction takes its A operand
// (m16n8k16, rows x K): a tile of 16 rows x 64 columns is 512 contiguous bytes, 16 per lane.  Lane
// 4 g + t holds four 32-bit words, word 2 c + h being columns 32 c + 8 t .. + 7 of row g + 8 h, and
// code j of a word sits in bits 4 (j / 2) + 16 (j % 2): two adjacent columns land in the two halves
// of a register after one AND, so a word gives four operand registers (columns 0-1, 2-3, 4-5, 6-7)
// for five integer instructions and a warp's loads are 512-byte runs.
#pragma once

#include <cuda_bf16.h>

#include "ifq_common.cuh"

namespace ifq {

constexpr int kQ4TileRows = 16, kQ4TileCols = 64, kQ4TileBytes = 512;

// A code n in bits 0-3 of a bf16 is the number n 2^-133 (a subnormal, since exponent fields 0 and 1
// share one spacing), and in bits 4-7 it is 16 n 2^-133.  One fused multiply-add per register turns
// both into (n - 8) 2^-6 or n 2^-6 exactly: multiplier 2^127 or 2^123, addend -2^-3 or 0.
constexpr uint32_t kQ4Mul0 = 0x7F007F00u;   // 2^127, twice
constexpr uint32_t kQ4Mul1 = 0x7D007D00u;   // 2^123
constexpr uint32_t kQ4Sub8 = 0xBE00BE00u;   // -2^-3 = -8 2^-6
constexpr float kQ4Unit = 64.0f;            // the 2^-6 of the operands, undone in float32

IFQ_DEVINL uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The four operand registers of a word: (n - 8) 2^-6 where kAdd = kQ4Sub8, n 2^-6 where it is -0.
template <uint32_t kAdd>
IFQ_DEVINL void q4_expand(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t v = w >> 8;
  a[0] = fma_bf16x2(w & 0x000F000Fu, kQ4Mul0, kAdd);
  a[1] = fma_bf16x2(w & 0x00F000F0u, kQ4Mul1, kAdd);
  a[2] = fma_bf16x2(v & 0x000F000Fu, kQ4Mul0, kAdd);
  a[3] = fma_bf16x2(v & 0x00F000F0u, kQ4Mul1, kAdd);
}

// D += A B, m16n8k16, bf16 operands, float32 accumulators.
IFQ_DEVINL void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B.
IFQ_DEVINL void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The 8 codes (0..15) of a word, from its columns' codes.
IFQ_DEVINL uint32_t q4_pack_word(const uint32_t (&n)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= n[j] << (4 * (j >> 1) + 16 * (j & 1));
  return w;
}

// q = rint(v / s) half-even of the exact quotient, for s > 0 a bf16 value and |v / s| below 2^20.  The
// product with a reciprocal may land one step off next to a half; the residual v - s q0 is exact in
// float32 (both are multiples of one unit and it is at most 1.5 s), so comparing it with s / 2 decides.
IFQ_DEVINL float q4_round_quotient(float v, float s, float inv) {
  const float q0 = rintf(s >= 1e-30f ? v * inv : v / s);
  const float f = fmaf(-s, q0, v);
  const float a = fabsf(f), h = 0.5f * s;
  const bool odd = ((int)q0 & 1) != 0;
  return (a > h || (a == h && odd)) ? q0 + copysignf(1.0f, f) : q0;
}

IFQ_DEVINL float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
IFQ_DEVINL float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
IFQ_DEVINL uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) |
         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi)) << 16);
}

IFQ_DEVINL void cp_async16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
IFQ_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
IFQ_DEVINL void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// 16 bytes that are read once, past L1.
IFQ_DEVINL uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

}  // namespace ifq

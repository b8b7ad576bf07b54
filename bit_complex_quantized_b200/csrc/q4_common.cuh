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

constexpr int kQ4TileBytes = 512;

// A code n in bits 0-3 of a bf16 is the number n 2^-133 (a subnormal, since exponent fields 0 and 1
// share one spacing), and in bits 4-7 it is 16 n 2^-133.  One fused multiply-add per register turns
// both into (n - 8) 2^-6 exactly: multiplier 2^127 or 2^123, addend -2^-3.
constexpr uint32_t kQ4Mul0 = 0x7F007F00u;   // 2^127, twice
constexpr uint32_t kQ4Mul1 = 0x7D007D00u;   // 2^123
constexpr uint32_t kQ4Sub8 = 0xBE00BE00u;   // -2^-3 = -8 2^-6
constexpr float kQ4Unit = 64.0f;            // the 2^-6 of the operands, undone in float32

IFQ_DEVINL uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The four operand registers of a word: (n - 8) 2^-6.
IFQ_DEVINL void q4_expand(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t v = w >> 8;
  a[0] = fma_bf16x2(w & 0x000F000Fu, kQ4Mul0, kQ4Sub8);
  a[1] = fma_bf16x2(w & 0x00F000F0u, kQ4Mul1, kQ4Sub8);
  a[2] = fma_bf16x2(v & 0x000F000Fu, kQ4Mul0, kQ4Sub8);
  a[3] = fma_bf16x2(v & 0x00F000F0u, kQ4Mul1, kQ4Sub8);
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

constexpr float kWideScale = 1e37f;  // 16 such steps are below the largest float32

// rint((x - m) / s) half-even of the exact quotient, clamped to [lo, hi], for finite x and bf16 values s > 0, m.
// d + e = x - m (two-term sum); the quotient of d decides except next to a half, where the residual d - s n
// (exact in float32: both are multiples of one unit and it is at most 1.5 s) plus e is compared with s / 2.
IFQ_DEVINL float exact_code(float x, float s, float m, float lo, float hi) {
  const float d = x - m;
  const float bb = d - x;
  const float e = (x - (d - bb)) - (m + bb);
  float n = fminf(fmaxf(rintf(d / s), lo), hi);
  const float f = fmaf(-s, n, d), h = 0.5f * s;
  const bool odd = ((int)n & 1) != 0;
  const float up = (f - h) + e, dn = (f + h) + e;
  if (up > 0.0f || (up == 0.0f && odd)) n += 1.0f;
  else if (dn < 0.0f || (dn == 0.0f && odd)) n -= 1.0f;
  return fminf(fmaxf(n, lo), hi);
}

// Two floats in a register pair, and arithmetic on both at once.
IFQ_DEVINL uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
IFQ_DEVINL uint64_t pair(float both) { return pair(both, both); }
IFQ_DEVINL float2 halves(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
IFQ_DEVINL uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
IFQ_DEVINL uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// Largest and smallest of three; NaN where one is NaN.
IFQ_DEVINL float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
IFQ_DEVINL float min3(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Four codes n_j = rint(kSpan r_j), r = a d + bias saturated to [0, 1], as the number n0 + 16 n1 + 256 n2 + 4096 n3 +
// base in bits 0-15 of the result.  kSpan r is within 2^-17 of the quotient that it stands for, so *near is set
// where that could decide the rounding (then exact_codes4 gives the answer).
template <int kSpan>
IFQ_DEVINL uint32_t fast_codes4(const float4& d, float a, float bias, float base, bool* near) {
  constexpr float kMagic = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer
  const uint64_t span = pair((float)kSpan), magic = pair(kMagic), minus = pair(-1.0f);
  const uint64_t r0 = pair(__saturatef(fmaf(d.x, a, bias)), __saturatef(fmaf(d.y, a, bias)));
  const uint64_t r1 = pair(__saturatef(fmaf(d.z, a, bias)), __saturatef(fmaf(d.w, a, bias)));
  const uint64_t n0 = fma2(fma2(r0, span, magic), minus, magic);  // -n
  const uint64_t n1 = fma2(fma2(r1, span, magic), minus, magic);
  const float2 e0 = halves(fma2(r0, span, n0)), e1 = halves(fma2(r1, span, n1));
  *near |= fmaxf(max3(fabsf(e0.x), fabsf(e0.y), fabsf(e1.x)), fabsf(e1.y)) > 0.49999f;
  const float2 u = halves(fma2(n1, pair(256.0f), n0));
  return __float_as_uint(fmaf(u.y, -16.0f, base + 8388608.0f) - u.x) & 0xFFFFu;
}
// v 2^-8, which keeps the sign of the smallest numbers: of those only the side of a half that they are on matters.
IFQ_DEVINL float shrink(float v) {
  const float r = v * 0.00390625f;
  return r == 0.0f && v != 0.0f ? copysignf(1.401298464e-45f, v) : r;
}
// The same by exact_code, code + base per entry; codes 0 where s = 0.  Where x - m may overflow (kMin: there is an m),
// all three are divided by 2^8 for large s.
template <bool kMin>
static __device__ __noinline__ uint32_t exact_codes4(float4 x, float s, float m, float lo, float hi, float base) {
  const float* f = &x.x;
  float sum = base;
  const bool wide = kMin && s > kWideScale;
  const float ss = wide ? shrink(s) : s, sm = wide ? shrink(m) : m;
#pragma unroll 1
  for (int j = 0; j < 4; ++j)
    sum += s > 0.0f ? exact_code(wide ? shrink(f[j]) : f[j], ss, sm, lo, hi) * (float)(1 << (4 * j)) : 0.0f;
  return (uint32_t)sum;
}
// A group's factor 1 / (span s) for fast_codes4 (0 where s = 0), and whether it is usable (not for scales so
// small that it overflows, or so large that x - m may).
template <bool kMin>
IFQ_DEVINL bool code_factor_usable(float s) {
  return s == 0.0f || (s >= 1e-30f && (!kMin || s <= kWideScale));
}
template <bool kMin>
IFQ_DEVINL float code_factor(float s, float inv_span, bool* usable) {
  *usable = code_factor_usable<kMin>(s);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // within 2^-23
  return s >= 1e-30f ? r * inv_span : 0.0f;
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

// The kernels of a decode step follow one another in a stream: each is launched while the one before ends, and reads and
// writes memory only when that one has ended (0.3 to 0.8 us a launch: appending and reading one token of 16 sequences
// 6.5 -> 5.6 us).  None lets the next one in earlier: its blocks would fill the places that are free first, and
// where a launch has no more blocks than the GPU has places they would crowd on some SMs (50021 x 4096 31.5 us against
// 25.8).
IFQ_DEVINL void follow() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Loads of what an earlier kernel may have written, for kernels that follow.  A load from the read-only path is one of
// constants to the compiler, which may move it in front of the wait, and promises nothing about lines that were fetched
// before they were written; these are ordinary loads, volatile so that they stay behind the wait.  (Through L2
// alone, past L1, appending and reading back 93 thousand tokens x heads takes 59 us against 50: every block looks up
// the same lengths and pages.)
IFQ_DEVINL int32_t ld_after(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
IFQ_DEVINL int64_t ld_after(const int64_t* p) {
  int64_t v;
  asm volatile("ld.global.s64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}
IFQ_DEVINL float2 ld_after(const float2* p) {
  float2 v;
  asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
IFQ_DEVINL int4 ld_after(const int4* p) {
  int4 v;
  asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// The address of such data as a value that is there behind the wait only: ordinary loads from it, in any order.
template <typename T>
IFQ_DEVINL T* behind_wait(T* p) {
  asm volatile("" : "+l"(p));
  return p;
}

template <typename P>
cudaError_t launch_following(void (*kernel)(P), dim3 grid, int threads, int smem, int cluster, const P& p,
                             cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// A kernel's shared memory above 48 KB has to be allowed once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, uint64_t* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (__atomic_load_n(done, __ATOMIC_ACQUIRE) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) __atomic_fetch_or(done, (uint64_t)1 << dev, __ATOMIC_RELEASE);
  return e;
}

// Everything that the cluster's CTAs did before is seen by all of them behind it.
IFQ_DEVINL void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

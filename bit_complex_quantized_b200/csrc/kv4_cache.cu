// The 4-bit key/value cache: new tokens in, stored values out.
//
// Each plane (real, imaginary) of a token's key or value of a head is one group: m = bf16(min),
// s = bf16(max c - min c), c the float32 nearest to 1/15 (float32 steps, nearest-even; two products, so
// that no range overflows), n = rint((x - m) / s) half-even of the exact quotient, clamped to [0, 15], 0 where s = 0.
// The stored value is s n + m.  Codes are chosen against the rounded s and m.
//
// A thread takes 8 entries; dim / 8 neighbouring threads hold a plane and reduce its minimum and
// maximum by shuffles.
#include "ifq_internal.h"
#include "kv4_common.cuh"

namespace ifq {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
  Kv4Arg c;
  const float* src[4];  // k_re, k_im, v_re, v_im
  float* dst[4];        // the same, for reading back
  int64_t ld;
  uint32_t* status;
};

constexpr float kBf16Max = 3.3895313892515355e38f;

// n = rint((x - m) / s), exact: d + e = x - m (two-term sum), the quotient of d decides except next to
// a half, where the residual d - s n0 (exact in float32) plus e is compared with s / 2.
IFQ_DEVINL uint32_t kv4_code(float x, float s, float m, float inv) {
  const float d = x - m;
  const float bb = d - x;
  const float e = (x - (d - bb)) - (m + bb);
  float n0 = rintf(s >= 1e-30f ? d * inv : d / s);
  n0 = fminf(fmaxf(n0, 0.0f), 15.0f);
  const float f = fmaf(-s, n0, d), h = 0.5f * s;
  const bool odd = ((int)n0 & 1) != 0;
  const float up = (f - h) + e, dn = (f + h) + e;   // f +- h is exact next to the half
  if (up > 0.0f || (up == 0.0f && odd)) n0 += 1.0f;
  else if (dn < 0.0f || (dn == 0.0f && odd)) n0 -= 1.0f;
  return (uint32_t)fminf(fmaxf(n0, 0.0f), 15.0f);
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LP = DIM / 8, D = 2 * DIM;
  const Kv4Arg& c = p.c;
  const int b = blockIdx.y;
  const Kv4Seq q = kv4_seq(c, b);
  if (!q.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
    return;
  }
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int part = (int)(idx % LP), plane = (int)(idx / LP) & 3;
  const int64_t th = idx / (4 * LP);
  const int head = (int)(th % c.kv_heads);
  const int64_t tok = th / c.kv_heads;
  const bool live = tok < q.n_new;
  float x[8] = {};
  bool bad = false;
  if (live) {
    const float4* src = reinterpret_cast<const float4*>(p.src[plane] + (q.row0 + tok) * p.ld + head * DIM + part * 8);
    const float4 a = __ldcs(src), bq = __ldcs(src + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = bq.x; x[5] = bq.y; x[6] = bq.z; x[7] = bq.w;
  }
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!(fabsf(x[j]) <= 3.402823466e38f)) {
      x[j] = 0.0f;
      bad = true;
    }
    x[j] = fminf(fmaxf(x[j], -kBf16Max), kBf16Max);
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
#pragma unroll
  for (int o = 1; o < LP; o *= 2) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!live) return;
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
  const __nv_bfloat16 mb = __float2bfloat16_rn(lo);
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fsub_rn(__fmul_rn(hi, 1.0f / 15.0f), __fmul_rn(lo, 1.0f / 15.0f)));
  const float s = __bfloat162float(sb), m = __bfloat162float(mb);
  const float inv = s >= 1e-30f ? __frcp_rn(s) : 0.0f;
  uint32_t n[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) n[j] = s > 0.0f ? kv4_code(x[j], s, m, inv) : 0u;

  const int32_t pos = q.len - q.n_new + (int32_t)tok;
  uint8_t* rec = kv4_record(c, b, head, pos >> 4);
  if (!rec) {
    if (part == 0) set_status(p.status, IFQ_DEV_RANGE);
    return;
  }
  const int r = pos & 15, hh = r >> 3;
  const int d = (plane & 1) * DIM + part * 8;  // first of the 8 stacked entries
  if (plane < 2) {
    uint32_t* w = reinterpret_cast<uint32_t*>(rec + (d >> 6) * 512 + (((r & 7) * 4 + ((d & 31) >> 3)) << 4));
    w[((d & 63) >> 5) * 2 + hh] = q4_pack_word(n);
  } else {
    const int qb = d >> 5, g = (d & 31) >> 2, t = (r & 7) >> 1;
    uint8_t* base = rec + 8 * D + (qb >> 1) * 512 + ((qb & 1) * 2 + hh) * 4 + (r & 1) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint16_t*>(base + (((g + i) * 4 + t) << 4)) =
          (uint16_t)(n[4 * i] | (n[4 * i + 1] << 4) | (n[4 * i + 2] << 8) | (n[4 * i + 3] << 12));
  }
  if (part == 0)
    *reinterpret_cast<uint32_t*>(rec + 16 * D + (plane >> 1) * 128 + r * 8 + (plane & 1) * 4) =
        (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(mb) << 16);
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LP = DIM / 8, D = 2 * DIM;
  const Kv4Arg& c = p.c;
  const int b = blockIdx.y;
  const Kv4Seq q = kv4_seq(c, b);
  if (!q.ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int part = (int)(idx % LP), plane = (int)(idx / LP) & 3;
  const int64_t th = idx / (4 * LP);
  const int head = (int)(th % c.kv_heads);
  const int64_t tok = th / c.kv_heads;
  if (tok >= q.n_new) return;
  float o[8] = {};
  uint8_t* rec = nullptr;
  const int32_t pos = q.len - q.n_new + (int32_t)tok;
  if (q.ok) {
    rec = kv4_record(c, b, head, pos >> 4);
    if (!rec && part == 0) set_status(p.status, IFQ_DEV_RANGE);
  }
  if (rec) {
    const int r = pos & 15, hh = r >> 3;
    const int d = (plane & 1) * DIM + part * 8;
    const uint32_t sm = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (plane >> 1) * 128 + r * 8 + (plane & 1) * 4);
    const float s = bf16_lo(sm), m = bf16_hi(sm);
    if (plane < 2) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(
          rec + (d >> 6) * 512 + (((r & 7) * 4 + ((d & 31) >> 3)) << 4))[((d & 63) >> 5) * 2 + hh];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(s, (float)((w >> (4 * (j >> 1) + 16 * (j & 1))) & 15u), m);
    } else {
      const int qb = d >> 5, g = (d & 31) >> 2, t = (r & 7) >> 1;
      const uint8_t* base = rec + 8 * D + (qb >> 1) * 512 + ((qb & 1) * 2 + hh) * 4 + (r & 1) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w = *reinterpret_cast<const uint16_t*>(base + (((g + i) * 4 + t) << 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) o[4 * i + j] = fmaf(s, (float)((w >> (4 * j)) & 15u), m);
      }
    }
  }
  float4* dst = reinterpret_cast<float4*>(p.dst[plane] + (q.row0 + tok) * p.ld + head * DIM + part * 8);
  __stcs(dst, make_float4(o[0], o[1], o[2], o[3]));
  __stcs(dst + 1, make_float4(o[4], o[5], o[6], o[7]));
}

template <int DIM>
cudaError_t launch(const AppendParams& p, bool read, cudaStream_t s) {
  const int64_t threads = (int64_t)p.c.n_new * p.c.kv_heads * (DIM / 2);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)p.c.B);
  if (read) kv4_read_kernel<DIM><<<grid, kThreads, 0, s>>>(p);
  else kv4_append_kernel<DIM><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t dispatch(const ifq_kv4_cache& c, const AppendParams& p, bool read, cudaStream_t s) {
  if (c.dim == 32) return launch<32>(p, read, s);
  if (c.dim == 64) return launch<64>(p, read, s);
  return launch<128>(p, read, s);
}

}  // namespace

cudaError_t launch_kv4_append(const ifq_kv4_cache& c, const float* k_re, const float* k_im, const float* v_re,
                              const float* v_im, int64_t ld, uint32_t* dev_status, cudaStream_t s) {
  AppendParams p = {kv4_arg(c), {k_re, k_im, v_re, v_im}, {}, ld, dev_status};
  return dispatch(c, p, false, s);
}

cudaError_t launch_kv4_read(const ifq_kv4_cache& c, float* k_re, float* k_im, float* v_re, float* v_im, int64_t ld,
                            uint32_t* dev_status, cudaStream_t s) {
  AppendParams p = {kv4_arg(c), {}, {k_re, k_im, v_re, v_im}, ld, dev_status};
  return dispatch(c, p, true, s);
}

}  // namespace ifq

// Layers with 4-bit weights and group scales: the quantizer and the values the codes stand for.
//
// For every group of G consecutive columns of a row of R: s = bf16(max |w| * c), c the float32 nearest
// to 1/7 (product in float32, both roundings to nearest-even), q = rint(w / s) half-even of the exact quotient, clamped
// to [-7, 7], 0 where s = 0; stored as q + 8.  Codes are chosen against the rounded scale, so the
// scale's rounding adds nothing to |w - s q| <= s / 2 but the clamp of a largest entry whose scale
// was rounded down (at most s 7 2^-9 more).
//
// HBM-bound: 4 bytes read and 0.5 + 2 / G written per weight.  Quantizing and dequantizing 10007 x 11008 in
// groups of 32 (723 MB) takes 118 us, 95 % of the copy rate, where the calls are captured in a graph, 137 us by calls one
// after the other; 4096 x 4096 (109 MB, two launches) 21.5 us, 79 %, and 25.6 us.  CTAs of 128 threads: of 256, two fit on
// an SM in groups of 128 (95 registers), 23.0 us captured.
// A warp takes 16 rows x max(64, G) columns, so that every group's maximum stays inside four lanes, loads are
// 32-byte runs per lane that fill whole 128-byte lines across a quad of lanes, and the codes leave as one
// 512-byte store per tile.
#include "ifq_internal.h"
#include "q4_common.cuh"

namespace ifq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct QArg {
  const float* R;
  uint8_t* codes;
  uint16_t* scales;
  uint16_t* out;  // dequantized bf16 [rows][cols]
  int64_t rows, cols;
  int64_t unit_begin;  // first unit (16 rows x U columns) of the tensor in the call
};

// Capacity kCap >= count: a launch copies its parameters, and most calls have few tensors.
template <int kCap>
struct QParams {
  QArg t[kCap];
  int count;
  int64_t units;
  uint32_t* status;
};

template <int kCap>
__device__ __forceinline__ int find_tensor(const QParams<kCap>& p, int64_t unit) {
  int i = 0;
  while (i + 1 < p.count && unit >= p.t[i + 1].unit_begin) ++i;
  return i;
}

template <int G, int kCap>
__global__ void __launch_bounds__(kThreads) w4_quant_kernel(const __grid_constant__ QParams<kCap> p) {
  constexpr int U = G > 64 ? G : 64, C = U / 32;      // columns and 32-column chunks of a unit
  constexpr int kPer = G / 32;                        // chunks of a group
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const QArg& T = p.t[find_tensor(p, unit)];
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t cu = T.cols / U, local = unit - T.unit_begin;
  const int64_t rt = local / cu, c0 = (local % cu) * U;

  float4 v[2][C][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = rt * 16 + g + 8 * h;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[h][c][i] = r < T.rows ? __ldcs(reinterpret_cast<const float4*>(T.R + r * T.cols + c0 + 32 * c + 8 * t) + i)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
  }

  bool bad = false;
  uint32_t words[2][C];
#pragma unroll
  for (int c0g = 0; c0g < C; c0g += kPer) {
    uint32_t sbits[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      auto largest = [&] {  // NaN or Inf with such a weight
        float m = 0.0f;
#pragma unroll
        for (int c = c0g; c < c0g + kPer; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4& x = v[h][c][i];
            m = max3(max3(m, fabsf(x.x), fabsf(x.y)), fabsf(x.z), fabsf(x.w));
          }
        return m;
      };
      float m = largest();
      if (!(m <= 3.402823466e38f)) {
        bad = true;
#pragma unroll
        for (int c = c0g; c < c0g + kPer; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* f = &v[h][c][i].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = fabsf(f[j]) <= 3.402823466e38f ? f[j] : 0.0f;
          }
        m = largest();
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(m, 1.0f / 7.0f));
      sbits[h] = __bfloat16_as_ushort(sb);
      const float s = __bfloat162float(sb);
      bool fast;
      const float factor = code_factor<false>(s, 1.0f / 14.0f, &fast);
      constexpr float kOnes = 1 + 16 + 256 + 4096;  // codes are stored plus 8; q + 7 = 14 (w / (14 s) + 1/2)
#pragma unroll
      for (int c = c0g; c < c0g + kPer; ++c) {
        const float4 &a = v[h][c][0], &b = v[h][c][1];
        uint32_t half[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // columns 0, 2, 4, 6 of the word, then 1, 3, 5, 7
          const float4 x = i == 0 ? make_float4(a.x, a.z, b.x, b.z) : make_float4(a.y, a.w, b.y, b.w);
          bool near = !fast;
          half[i] = fast_codes4<14>(x, factor, 0.5f, kOnes, &near);
          if (near) half[i] = exact_codes4<false>(x, s, 0.0f, -7.0f, 7.0f, 8.0f * kOnes);
        }
        words[h][c] = half[0] | (half[1] << 16);
      }
    }
    if (t == 0)
      reinterpret_cast<uint32_t*>(T.scales)[(rt * (T.cols / G) + (c0 + 32 * c0g) / G) * 8 + g] =
          sbits[0] | (sbits[1] << 16);
  }
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
#pragma unroll
  for (int k = 0; k < C / 2; ++k) {
    uint4 w = make_uint4(words[0][2 * k], words[1][2 * k], words[0][2 * k + 1], words[1][2 * k + 1]);
    reinterpret_cast<uint4*>(T.codes)[(rt * (T.cols / 64) + c0 / 64 + k) * 32 + lane] = w;
  }
}

template <int G, int kCap>
__global__ void __launch_bounds__(kThreads) w4_dequant_kernel(const __grid_constant__ QParams<kCap> p) {
  constexpr int U = G > 64 ? G : 64;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const QArg& T = p.t[find_tensor(p, unit)];
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t cu = T.cols / U, local = unit - T.unit_begin;
  const int64_t rt = local / cu, c0 = (local % cu) * U;
  uint4 w[U / 64];
#pragma unroll
  for (int k = 0; k < U / 64; ++k)
    w[k] = ldg_stream(reinterpret_cast<const uint4*>(T.codes) + (rt * (T.cols / 64) + c0 / 64 + k) * 32 + lane);
#pragma unroll
  for (int k = 0; k < U / 64; ++k)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t sc = __ldg(reinterpret_cast<const uint32_t*>(T.scales) +
                                (rt * (T.cols / G) + (c0 + 64 * k + 32 * c) / G) * 8 + g);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t r = rt * 16 + g + 8 * h;
        const float s = h ? bf16_hi(sc) : bf16_lo(sc);
        const uint32_t word = c ? (h ? w[k].w : w[k].z) : (h ? w[k].y : w[k].x);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = (float)((int)((word >> (4 * i)) & 15u) - 8);
          const float hi = (float)((int)((word >> (4 * i + 16)) & 15u) - 8);
          o[i] = pack_bf16(s * lo, s * hi);
        }
        if (r < T.rows)
          __stcs(reinterpret_cast<uint4*>(T.out + r * T.cols + c0 + 64 * k + 32 * c + 8 * t),
                 make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
}

enum class Op { kQuantize, kDequantize };

template <Op kOp, int G, int kCap>
void run(const QParams<kCap>& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.units + kWarps - 1) / kWarps);
  if constexpr (kOp == Op::kQuantize) w4_quant_kernel<G, kCap><<<grid, kThreads, 0, s>>>(p);
  else w4_dequant_kernel<G, kCap><<<grid, kThreads, 0, s>>>(p);
}

// arg(i): the i-th tensor's pointers and sizes.
template <Op kOp, int kCap, typename Arg>
cudaError_t launch(int count, int group, uint32_t* dev_status, cudaStream_t s, Arg arg) {
  QParams<kCap> p;
  p.count = count;
  p.status = dev_status;
  p.units = 0;
  for (int i = 0; i < count; ++i) {
    p.t[i] = arg(i);
    p.t[i].unit_begin = p.units;
    p.units += w4_units(p.t[i].rows, p.t[i].cols, group);
  }
  if (group == 32) run<kOp, 32>(p, s);
  else if (group == 64) run<kOp, 64>(p, s);
  else run<kOp, 128>(p, s);
  return cudaGetLastError();
}

}  // namespace

int64_t w4_units(int64_t rows, int64_t cols, int group) {
  return (rows + 15) / 16 * (cols / (group > 64 ? group : 64));
}

cudaError_t launch_w4_quantize(const ifq_w4_tensor* ts, int count, int group, uint32_t* dev_status, cudaStream_t s) {
  auto arg = [&](int i) { return QArg{ts[i].R, ts[i].codes, ts[i].scales, nullptr, ts[i].rows, ts[i].cols, 0}; };
  return count <= 8 ? launch<Op::kQuantize, 8>(count, group, dev_status, s, arg)
                    : launch<Op::kQuantize, IFQ_MAX_GROUP>(count, group, dev_status, s, arg);
}

cudaError_t launch_w4_dequantize(const ifq_w4_dqtensor* ts, int count, int group, cudaStream_t s) {
  auto arg = [&](int i) {
    return QArg{nullptr, const_cast<uint8_t*>(ts[i].codes), const_cast<uint16_t*>(ts[i].scales), ts[i].w, ts[i].rows,
                ts[i].cols, 0};
  };
  return count <= 8 ? launch<Op::kDequantize, 8>(count, group, nullptr, s, arg)
                    : launch<Op::kDequantize, IFQ_MAX_GROUP>(count, group, nullptr, s, arg);
}

}  // namespace ifq

// Decode product of layers with 4-bit weights and group scales, y = R_hat [x_re; x_im] for 1 to 16
// tokens: y[n][r] = sum_groups s[r][group] sum_{k in group} q[r][k] x[n][k].
//
// Each 32-bit word of eight codes becomes four bf16 operand registers holding q 2^-6 exactly
// (q4_common.cuh), x is the B operand as it is, so all products are exact and a group accumulates
// in float32; the group's scale multiplies that sum in float32.
#include "ifq_internal.h"
#include "q4_common.cuh"

namespace ifq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = kWarps * 16;  // rows of a CTA

struct LArg {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* x[2];
  float* y[2];
  int64_t rows, cols;
  int64_t x_split, y_split;  // first column / row of the second plane (cols / rows where there is none)
  int64_t tile_begin;
};

struct LParams {
  LArg l[IFQ_MAX_GROUP];
  int count, B;
  uint32_t* status;
};

template <int G, int NT>
__global__ void __launch_bounds__(kThreads) w4_gemv_kernel(const __grid_constant__ LParams p) {
  constexpr int U = G > 64 ? G : 64;
  int li = 0;
  while (li + 1 < p.count && (int64_t)blockIdx.x >= p.l[li + 1].tile_begin) ++li;
  const LArg& L = p.l[li];
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t rt = ((int64_t)blockIdx.x - L.tile_begin) * kWarps + (threadIdx.x >> 5);
  if (rt * 16 >= L.rows) return;
  float acc[NT][4] = {};
  const uint4* codes = reinterpret_cast<const uint4*>(L.codes) + rt * (L.cols / 64) * 32 + lane;
  const uint32_t* scales = reinterpret_cast<const uint32_t*>(L.scales) + rt * (L.cols / G) * 8 + g;
  for (int64_t k0 = 0; k0 < L.cols; k0 += U) {
    float part[NT][4] = {};
#pragma unroll
    for (int i = 0; i < U / 64; ++i) {
      const uint4 w4 = ldg_stream(codes + (k0 / 64 + i) * 32);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t k = k0 + 64 * i + 32 * c;
        const int pl = k >= L.x_split;
        const int64_t width = pl ? L.cols - L.x_split : L.x_split;
        uint32_t lo[4], hi[4];
        q4_expand<kQ4Sub8>(w[2 * c], lo);
        q4_expand<kQ4Sub8>(w[2 * c + 1], hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint4 b = make_uint4(0, 0, 0, 0);
          if (nt * 8 + g < p.B)
            b = __ldg(reinterpret_cast<const uint4*>(L.x[pl] + (nt * 8 + g) * width + (k - (pl ? L.x_split : 0)) + 8 * t));
          mma_bf16(part[nt], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
          mma_bf16(part[nt], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
        }
        if ((64 * i + 32 * c + 32) % G == 0) {
          const uint32_t sc = __ldg(scales + (k / G) * 8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] += bf16_lo(sc) * part[nt][0];
            acc[nt][1] += bf16_lo(sc) * part[nt][1];
            acc[nt][2] += bf16_hi(sc) * part[nt][2];
            acc[nt][3] += bf16_hi(sc) * part[nt][3];
            part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.0f;
          }
        }
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t r = rt * 16 + g + 8 * (e >> 1);
      const int n = nt * 8 + 2 * t + (e & 1);
      if (r >= L.rows || n >= p.B) continue;
      const float v = acc[nt][e] * kQ4Unit;
      bad |= !(fabsf(v) <= 3.402823466e38f);
      if (r < L.y_split) L.y[0][n * L.y_split + r] = v;
      else L.y[1][n * (L.rows - L.y_split) + r - L.y_split] = v;
    }
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
}

template <int G>
cudaError_t launch(const LParams& p, int64_t tiles, cudaStream_t s) {
  if (p.B <= 8) w4_gemv_kernel<G, 1><<<(unsigned)tiles, kThreads, 0, s>>>(p);
  else w4_gemv_kernel<G, 2><<<(unsigned)tiles, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_w4_gemv(const ifq_w4_layer* Ls, int count, int group, int B, uint32_t* dev_status, cudaStream_t s) {
  LParams p = {};
  p.count = count;
  p.B = B;
  p.status = dev_status;
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i) {
    const ifq_w4_layer& a = Ls[i];
    LArg& l = p.l[i];
    l.codes = a.codes;
    l.scales = a.scales;
    l.x[0] = a.x_re;
    l.x[1] = a.x_im;
    l.y[0] = a.y_re;
    l.y[1] = a.y_im;
    l.rows = a.rows;
    l.cols = a.cols;
    l.x_split = a.x_im ? a.cols / 2 : a.cols;
    l.y_split = a.y_im ? a.rows / 2 : a.rows;
    l.tile_begin = tiles;
    tiles += (a.rows + kRows - 1) / kRows;
  }
  if (group == 32) return launch<32>(p, tiles, s);
  if (group == 64) return launch<64>(p, tiles, s);
  return launch<128>(p, tiles, s);
}

}  // namespace ifq

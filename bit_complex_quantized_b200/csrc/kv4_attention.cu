// Decode attention over the 4-bit key/value cache: for each query head of each new token
//   score_j = scale (q_re . k_re,j + q_im . k_im,j),  o = sum_j softmax(score)_j v_j,
// keys j <= the token's position, o's planes summed separately.
//
// One pass over the cache with the running maximum and sum of the softmax.  A warp takes 32 keys at a
// time (two records): keys are the rows of the matrix instruction's A operand, queries the columns of B.
//   q     float32, times scale log2 e, split into two bf16 terms (high, low: 2^-16 relative) that
//         are two neighbouring columns, so that the scores keep float32's order of accuracy
//   K     codes minus 8, exact; s and m of a key's plane enter per score in float32:
//         score = sum_planes s (codes . q) + (m + 8 s) sum(q)
//   P     p s per key and plane, split the same way, transposed in registers (movmatrix) from the
//         score layout into the B operand; o = sum_j (p s)_j codes_j + sum_j p_j (m + 8 s)_j
// A product of a column pair is added up within one lane.
#include "ifq_internal.h"
#include "kv4_common.cuh"

namespace ifq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;                  // keys of a warp's step
constexpr int kBlockKeys = kWarps * kStep;
constexpr int kMaxSplits = 64;

struct AttnParams {
  Kv4Arg c;
  const float* q[2];
  uint16_t* o[2];
  int64_t ldq, ldo;
  float scale2;      // scale log2 e
  int32_t shared;    // query heads of a key/value head
  int32_t splits, qtiles;
  float* ws_o;       // [B][kv_heads][qtiles QR][splits][D]
  float2* ws_ml;     // [B][kv_heads][qtiles QR][splits]: maximum (log2), sum
  uint32_t* status;
};

IFQ_DEVINL float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 x 8 transpose of 16-bit elements over a warp.
IFQ_DEVINL uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// v as two bf16 terms, the larger in the low half.
IFQ_DEVINL uint32_t split_bf16(float v) {
  const float hi = __bfloat162float(__float2bfloat16_rn(v));
  return pack_bf16(hi, v - hi);
}

// Keys of a split of a sequence of len keys: whole blocks, shared evenly.
IFQ_DEVINL int32_t split_keys(int32_t len, int32_t splits) {
  const int32_t blocks = (len + kBlockKeys - 1) / kBlockKeys;
  return (blocks + splits - 1) / splits * kBlockKeys;
}

template <int DIM, int NT>
__global__ void __launch_bounds__(kThreads) kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  constexpr int D = 2 * DIM, CH = D / 32, CP = DIM / 32, QR = 4 * NT, T4 = D / 64;
  __shared__ uint4 qs[NT][CH][32];          // B operands of q
  __shared__ float qsum[QR][2];             // sum of a query's plane
  __shared__ float os[kWarps][QR][D];
  __shared__ float2 mls[kWarps][QR];
  const Kv4Arg& c = p.c;
  const int b = blockIdx.z, kvh = blockIdx.y / p.qtiles, qt = blockIdx.y % p.qtiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Kv4Seq sq = kv4_seq(c, b);
  if (!sq.ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
  const int nrows = sq.n_new * p.shared - qt * QR;  // query rows of this tile
  if (nrows <= 0) return;
  const int32_t per = split_keys(sq.len, p.splits);
  const int32_t k_begin = (int32_t)blockIdx.x * per;
  const int32_t k_end = min(sq.len, k_begin + per);
  if (blockIdx.x > 0 && k_begin >= k_end) return;

  // q: thread (nt, ch, lane) of the operand order
  for (int i = threadIdx.x; i < NT * CH * 32; i += kThreads) {
    const int ln = i & 31, ch = (i >> 5) % CH, nt = (i >> 5) / CH;
    const int row = nt * 4 + (ln >> 3), part = (ln >> 2) & 1;
    uint32_t w[4] = {};
    if (row < nrows) {
      const int rr = qt * QR + row, tok = rr / p.shared, head = kvh * p.shared + rr % p.shared;
      const int d = ch * 32 + (ln & 3) * 8;
      const float* src = p.q[d / DIM] + (sq.row0 + tok) * p.ldq + head * DIM + d % DIM;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(src) + j);
        const uint32_t a = split_bf16(v.x * p.scale2), bq = split_bf16(v.y * p.scale2);
        w[j] = part ? (a >> 16) | (bq & 0xFFFF0000u) : (a & 0xFFFFu) | (bq << 16);
        if (!(fabsf(v.x) <= 3.402823466e38f) || !(fabsf(v.y) <= 3.402823466e38f))
          set_status(p.status, IFQ_DEV_NONFINITE);
      }
    }
    qs[nt][ch][ln] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < QR * 2; i += kThreads) {
    const int row = i >> 1, pl = i & 1;
    float sum = 0.0f;
    for (int ch = pl * CP; ch < (pl + 1) * CP; ++ch)
      for (int l = 0; l < 8; ++l) {
        const uint4 v = qs[row >> 2][ch][(row & 3) * 8 + l];
        sum += (bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y)) + (bf16_lo(v.z) + bf16_hi(v.z)) +
               (bf16_lo(v.w) + bf16_hi(v.w));
      }
    qsum[row][pl] = sum;
  }
  __syncthreads();

  float qs2[NT][2];
  int32_t visible[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = nt * 4 + t;
    qs2[nt][0] = qsum[row][0];
    qs2[nt][1] = qsum[row][1];
    visible[nt] = row < nrows ? sq.len - sq.n_new + (qt * QR + row) / p.shared + 1 : 0;
  }

  float acc[CH][2][NT][4];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[i][j][nt][0] = acc[i][j][nt][1] = acc[i][j][nt][2] = acc[i][j][nt][3] = 0.0f;
  float m_run[NT], l_run[NT], pm[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_run[nt] = -INFINITY;
    l_run[nt] = pm[nt][0] = pm[nt][1] = 0.0f;
  }

  for (int32_t key0 = k_begin + warp * kStep; key0 < k_end; key0 += kBlockKeys) {
    const uint8_t* rec[2];
    float sc[2][NT][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t kt = key0 + 16 * i;
      rec[i] = kt < k_end ? kv4_record(c, b, kvh, kt >> 4) : nullptr;
      if (kt < k_end && !rec[i] && lane == 0) set_status(p.status, IFQ_DEV_RANGE);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[i][nt][0] = sc[i][nt][1] = -INFINITY;
      if (!rec[i]) continue;
      float s4[2][NT][4] = {};
#pragma unroll
      for (int v = 0; v < T4; ++v) {
        const uint4 w4 = ldg_stream(rec[i] + v * 512 + lane * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int ch = 2 * v + cc, pl = ch / CP;
          uint32_t lo[4], hi[4];
          q4_expand<kQ4Sub8>(w[2 * cc], lo);
          q4_expand<kQ4Sub8>(w[2 * cc + 1], hi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 bq = qs[nt][ch][lane];
            mma_bf16(s4[pl][nt], lo[0], hi[0], lo[1], hi[1], bq.x, bq.y);
            mma_bf16(s4[pl][nt], lo[2], hi[2], lo[3], hi[3], bq.z, bq.w);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 par = __ldg(reinterpret_cast<const uint2*>(rec[i] + 16 * D + (g + 8 * h) * 8));
        const float s0 = bf16_lo(par.x), m0 = fmaf(8.0f, s0, bf16_hi(par.x));
        const float s1 = bf16_lo(par.y), m1 = fmaf(8.0f, s1, bf16_hi(par.y));
        const float u0 = s0 * kQ4Unit, u1 = s1 * kQ4Unit;
        const int32_t key = kt + g + 8 * h;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float a0 = s4[0][nt][2 * h] + s4[0][nt][2 * h + 1], a1 = s4[1][nt][2 * h] + s4[1][nt][2 * h + 1];
          const float v = fmaf(u0, a0, m0 * qs2[nt][0]) + fmaf(u1, a1, m1 * qs2[nt][1]);
          sc[i][nt][h] = key < visible[nt] ? v : -INFINITY;
        }
      }
    }
    float mb[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx = fmaxf(fmaxf(sc[0][nt][0], sc[0][nt][1]), fmaxf(sc[1][nt][0], sc[1][nt][1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float mn = fmaxf(m_run[nt], mx);
      mb[nt] = mn == -INFINITY ? 0.0f : mn;
      const float al = ex2(m_run[nt] - mb[nt]);
      m_run[nt] = mn;
      l_run[nt] *= al;
      pm[nt][0] *= al;
      pm[nt][1] *= al;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][nt][e] *= al;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!rec[i]) continue;
      uint32_t pb[2][NT][2];  // B operands of p s: plane, n tile, keys 0-7 / 8-15
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 par = __ldg(reinterpret_cast<const uint2*>(rec[i] + 16 * D + 128 + (g + 8 * h) * 8));
        const float s0 = bf16_lo(par.x), m0 = fmaf(8.0f, s0, bf16_hi(par.x));
        const float s1 = bf16_lo(par.y), m1 = fmaf(8.0f, s1, bf16_hi(par.y));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float pr = ex2(sc[i][nt][h] - mb[nt]);
          l_run[nt] += pr;
          // rows behind the last key hold whatever the page held: their weight is zero, not their product
          const bool on = sc[i][nt][h] != -INFINITY;
          pm[nt][0] += on ? pr * m0 : 0.0f;
          pm[nt][1] += on ? pr * m1 : 0.0f;
          pb[0][nt][h] = movmatrix(on ? split_bf16(pr * s0) : 0u);
          pb[1][nt][h] = movmatrix(on ? split_bf16(pr * s1) : 0u);
        }
      }
#pragma unroll
      for (int v = 0; v < T4; ++v) {
        const uint4 w4 = ldg_stream(rec[i] + 8 * D + v * 512 + lane * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int ch = 2 * v + cc, pl = ch / CP;
          uint32_t lo[4], hi[4];
          q4_expand<kQ4Sub8>(w[2 * cc], lo);
          q4_expand<kQ4Sub8>(w[2 * cc + 1], hi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(acc[ch][0][nt], lo[0], lo[1], hi[0], hi[1], pb[pl][nt][0], pb[pl][nt][1]);
            mma_bf16(acc[ch][1][nt], lo[2], lo[3], hi[2], hi[3], pb[pl][nt][0], pb[pl][nt][1]);
          }
        }
      }
    }
  }

  // the warps' parts, then their sum
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int o = 4; o < 32; o *= 2) {
      l_run[nt] += __shfl_xor_sync(0xffffffffu, l_run[nt], o);
      pm[nt][0] += __shfl_xor_sync(0xffffffffu, pm[nt][0], o);
      pm[nt][1] += __shfl_xor_sync(0xffffffffu, pm[nt][1], o);
    }
    const int row = nt * 4 + t;
    if (g == 0) mls[warp][row] = make_float2(m_run[nt], l_run[nt]);
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      const float pmv = pm[nt][ch / CP];
      float4 v;
      v.x = fmaf(kQ4Unit, acc[ch][0][nt][0] + acc[ch][0][nt][1], pmv);
      v.y = fmaf(kQ4Unit, acc[ch][0][nt][2] + acc[ch][0][nt][3], pmv);
      v.z = fmaf(kQ4Unit, acc[ch][1][nt][0] + acc[ch][1][nt][1], pmv);
      v.w = fmaf(kQ4Unit, acc[ch][1][nt][2] + acc[ch][1][nt][3], pmv);
      *reinterpret_cast<float4*>(&os[warp][row][ch * 32 + 4 * g]) = v;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < QR * (D / 2); i += kThreads) {
    const int row = i / (D / 2), d = (i % (D / 2)) * 2;
    if (row >= nrows) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mls[w][row].x);
    const float ms = M == -INFINITY ? 0.0f : M;
    float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(mls[w][row].x - ms);
      l += f * mls[w][row].y;
      o0 += f * os[w][row][d];
      o1 += f * os[w][row][d + 1];
    }
    const int rr = qt * QR + row;
    if (p.splits == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int tok = rr / p.shared, head = kvh * p.shared + rr % p.shared;
      *reinterpret_cast<uint32_t*>(p.o[d / DIM] + (sq.row0 + tok) * p.ldo + head * DIM + d % DIM) =
          pack_bf16(o0 * inv, o1 * inv);
    } else {
      const int64_t at = ((((int64_t)b * c.kv_heads + kvh) * p.qtiles * QR) + rr) * p.splits + blockIdx.x;
      *reinterpret_cast<float2*>(p.ws_o + at * D + d) = make_float2(o0, o1);
      if (d == 0) p.ws_ml[at] = make_float2(M, l);
    }
  }
}

// The splits of a query row, added in their order.  One warp per query row.
template <int DIM>
__global__ void __launch_bounds__(kThreads) kv4_merge_kernel(const __grid_constant__ AttnParams p, int qr) {
  constexpr int D = 2 * DIM;
  const Kv4Arg& c = p.c;
  const int lane = threadIdx.x & 31, b = blockIdx.z, kvh = blockIdx.y;
  const int rr = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const Kv4Seq sq = kv4_seq(c, b);
  if (rr >= sq.n_new * p.shared) return;
  const int32_t per = split_keys(sq.len, p.splits);
  const int used = sq.len > 0 ? (sq.len + per - 1) / per : 1;
  const int64_t at = (((int64_t)b * c.kv_heads + kvh) * p.qtiles * qr + rr) * p.splits;
  float M = -INFINITY;
  for (int s = 0; s < used; ++s) M = fmaxf(M, p.ws_ml[at + s].x);
  const float ms = M == -INFINITY ? 0.0f : M;
  float l = 0.0f;
  float2 o[D / 64] = {};
  for (int s = 0; s < used; ++s) {
    const float2 ml = p.ws_ml[at + s];
    const float f = ex2(ml.x - ms);
    l += f * ml.y;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(p.ws_o + (at + s) * D + i * 64 + lane * 2);
      o[i].x += f * v.x;
      o[i].y += f * v.y;
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = rr / p.shared, head = kvh * p.shared + rr % p.shared;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int d = i * 64 + lane * 2;
    *reinterpret_cast<uint32_t*>(p.o[d / DIM] + (sq.row0 + tok) * p.ldo + head * DIM + d % DIM) =
        pack_bf16(o[i].x * inv, o[i].y * inv);
  }
}

struct Plan {
  int nt, qtiles, splits;
};

// Two n tiles (8 query rows) where there are more than 4 query rows; as many splits as fill the GPU.
Plan plan(const ifq_kv4_cache& c, int shared) {
  Plan r;
  const int64_t rows = (int64_t)c.n_new * shared;
  r.nt = rows > 4 ? 2 : 1;
  r.qtiles = (int)((rows + 4 * r.nt - 1) / (4 * r.nt));
  const int64_t ctas = (int64_t)c.B * c.kv_heads * r.qtiles;
  const int64_t blocks = (c.table_cols * c.page_tokens + kBlockKeys - 1) / kBlockKeys;
  int64_t s = (148 * 4 + ctas - 1) / ctas;
  if (s > blocks) s = blocks;
  if (s > kMaxSplits) s = kMaxSplits;
  r.splits = s < 1 ? 1 : (int)s;
  return r;
}

int64_t partials(const ifq_kv4_cache& c, const Plan& r) {
  return (int64_t)c.B * c.kv_heads * r.qtiles * 4 * r.nt * r.splits;
}

template <int DIM>
cudaError_t launch(const AttnParams& p, const Plan& r, cudaStream_t s) {
  const dim3 grid((unsigned)r.splits, (unsigned)(p.c.kv_heads * r.qtiles), (unsigned)p.c.B);
  if (r.nt == 1) kv4_attn_kernel<DIM, 1><<<grid, kThreads, 0, s>>>(p);
  else kv4_attn_kernel<DIM, 2><<<grid, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || r.splits == 1) return e;
  const dim3 mg((unsigned)((p.c.n_new * p.shared + kWarps - 1) / kWarps), (unsigned)p.c.kv_heads, (unsigned)p.c.B);
  kv4_merge_kernel<DIM><<<mg, kThreads, 0, s>>>(p, 4 * r.nt);
  return cudaGetLastError();
}

}  // namespace

size_t kv4_attention_workspace_bytes(const ifq_kv4_cache& c, int shared) {
  const Plan r = plan(c, shared);
  if (r.splits == 1) return 0;
  return (size_t)partials(c, r) * (2 * c.dim + 2) * 4;
}

cudaError_t launch_kv4_attention(const ifq_kv4_cache& c, int shared, const float* q_re, const float* q_im, int64_t ldq,
                                 float scale, uint16_t* o_re, uint16_t* o_im, int64_t ldo, void* ws,
                                 uint32_t* dev_status, cudaStream_t s) {
  const Plan r = plan(c, shared);
  AttnParams p = {};
  p.c = kv4_arg(c);
  p.q[0] = q_re;
  p.q[1] = q_im;
  p.o[0] = o_re;
  p.o[1] = o_im;
  p.ldq = ldq;
  p.ldo = ldo;
  p.scale2 = scale * 1.4426950408889634f;
  p.shared = shared;
  p.splits = r.splits;
  p.qtiles = r.qtiles;
  p.ws_o = static_cast<float*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(static_cast<float*>(ws) + partials(c, r) * 2 * c.dim);
  p.status = dev_status;
  if (c.dim == 32) return launch<32>(p, r, s);
  if (c.dim == 64) return launch<64>(p, r, s);
  return launch<128>(p, r, s);
}

}  // namespace ifq

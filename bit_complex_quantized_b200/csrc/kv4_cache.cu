// The 4-bit key/value cache: new tokens in, stored values out.
//
// Each plane (real, imaginary) of a token's key or value of a head is one group: m = bf16(min),
// s = bf16(max c - min c), c the float32 nearest to 1/15 (float32 steps, nearest-even; two products, so
// that no range overflows), n = rint((x - m) / s) half-even of the exact quotient, clamped to [0, 15], 0 where s = 0.
// The stored value is s n + m.  Codes are chosen against the rounded s and m.
//
// Two forms, by the new tokens of a sequence.
//   fewer than 16 (decode)  a thread takes 8 entries of a token, dim / 8 neighbouring threads a plane, and writes its
//           words and half words alone: as many threads as there are entries, the shortest chain.  16 sequences of
//           8 heads: appending takes 2.6 us, with reading back 5.1 us (captured), against 26.6 us by records (a warp
//           then has one live token of 16 in a chain 16 times as long).
//   16 and more (prompts)   a warp takes one plane of a record (16 tokens of a head) and then the next heads' (up to 8,
//           so that lengths, pages and places are found once): keys as lane (g, t) holds them
//           in the record (8 entries of the tokens g and g + 8 per 32 columns), values likewise (4 entries of
//           four tokens), so that loads are 128-byte runs, and a record that is all new leaves as 512-byte stores.
//           The lanes of a plane share out its minima and maxima as they join them, so each makes one group's
//           parameters.  A record that holds older tokens
//           too is written token by token: a token's keys are whole words and its values whole half words, so
//           nothing is read back.  93 thousand tokens x heads of dim 64, appending and reading back: 44 us (203 MB,
//           4.6 TB/s), against 149 us by tokens (scattered 2 and 4 byte stores).
// HBM-bound in bytes (16 dim read and 2 dim + 16 written per token and head): 20000 tokens of 32 heads are appended in
// 122 us, 95 % of the copy rate (131 us without the prefetch of the next head), 93 thousand tokens x heads in 24 us, 70 %.
#include "ifq_internal.h"
#include "kv4_common.cuh"

namespace ifq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

struct AppendParams {
  Kv4Arg c;
  const float* src[4];  // k_re, k_im, v_re, v_im
  float* dst[4];        // the same, for reading back
  int64_t ld;
  int32_t heads_each;   // heads that a CTA appends one after the other
  uint32_t* status;
};

constexpr float kBf16Max = 3.3895313892515355e38f;

// The record of a warp: its address (null: none), its first position, the sequence.
struct Item {
  uint8_t* rec;
  int32_t pos0, first;  // position of the record's token 0; first new position
  Kv4Seq q;
  int head;
};

// Record `tile` (counted from the first that the new tokens touch) of head `head` of sequence blockIdx.z.
IFQ_DEVINL bool find_item(const AppendParams& p, const Kv4Seq& q, int32_t tile, int head, Item* it) {
  if (q.n_new == 0) return false;  // its last record holds no token of the call: its page is not looked up
  it->q = q;
  it->head = head;
  // a sequence whose length is unusable has no positions, but its rows still read as 0
  const int32_t len = q.ok ? q.len : q.n_new;
  it->first = len - q.n_new;
  tile += it->first >> 4;
  if ((int64_t)tile * 16 >= len) return false;
  it->pos0 = tile * 16;
  it->rec = nullptr;
  if (q.ok) {
    it->rec = kv4_record(p.c, blockIdx.z, head, tile);
    if (!it->rec && (threadIdx.x & 31) == 0) set_status(p.status, IFQ_DEV_RANGE);
  }
  return true;
}

struct Group {  // a plane's parameters
  float s, m, factor;
  uint32_t bits;
  bool fast;
};
IFQ_DEVINL Group group_of(float lo, float hi) {
  const __nv_bfloat16 mb = __float2bfloat16_rn(lo);
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fsub_rn(__fmul_rn(hi, 1.0f / 15.0f), __fmul_rn(lo, 1.0f / 15.0f)));
  Group r;
  r.s = __bfloat162float(sb);
  r.m = __bfloat162float(mb);
  r.factor = code_factor<true>(r.s, 1.0f / 15.0f, &r.fast);
  r.bits = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(mb) << 16);
  return r;
}
// The group that lane `from` of the warp holds.
IFQ_DEVINL Group group_from(const Group& own, int from) {
  Group r;
  r.bits = __shfl_sync(0xffffffffu, own.bits, from);
  r.factor = __shfl_sync(0xffffffffu, own.factor, from);
  r.s = bf16_lo(r.bits);
  r.m = bf16_hi(r.bits);
  r.fast = code_factor_usable<true>(r.s);
  return r;
}
// Minima and maxima of two groups, over lanes that differ in bit `mask`: the lane whose bit is set goes on with the
// second group, the other with the first.
IFQ_DEVINL void halve(float lo0, float lo1, float hi0, float hi1, int mask, bool second, float* lo, float* hi) {
  *lo = fminf(second ? lo1 : lo0, __shfl_xor_sync(0xffffffffu, second ? lo0 : lo1, mask));
  *hi = fmaxf(second ? hi1 : hi0, __shfl_xor_sync(0xffffffffu, second ? hi0 : hi1, mask));
}
IFQ_DEVINL void both(float* lo, float* hi, int mask) {
  *lo = fminf(*lo, __shfl_xor_sync(0xffffffffu, *lo, mask));
  *hi = fmaxf(*hi, __shfl_xor_sync(0xffffffffu, *hi, mask));
}
// Entry j of four in bits 4 j.
IFQ_DEVINL uint32_t codes_of(const float4& x, const Group& q) {
  bool near = !q.fast;
  const uint64_t minus_m = pair(-q.m);
  const float2 d0 = halves(add2(pair(x.x, x.y), minus_m)), d1 = halves(add2(pair(x.z, x.w), minus_m));
  const float4 d = make_float4(d0.x, d0.y, d1.x, d1.y);
  const uint32_t w = fast_codes4<15>(d, q.factor, 0.0f, 0.0f, &near);
  return near ? exact_codes4<true>(x, q.s, q.m, 0.0f, 15.0f, 0.0f) : w;
}
// The word of eight entries of a key: entries 0, 2, 4, 6 in the low half, 1, 3, 5, 7 in the high half.
IFQ_DEVINL uint32_t key_word(const float4& a, const float4& b, const Group& q) {
  return codes_of(make_float4(a.x, a.z, b.x, b.z), q) | (codes_of(make_float4(a.y, a.w, b.y, b.w), q) << 16);
}

// src: from behind_wait.
IFQ_DEVINL float4 take(const float* src, bool in) {
  return in ? __ldcs(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
}
// Minimum and maximum so far, NaN with a NaN entry.
IFQ_DEVINL void widen(const float4& v, float* lo, float* hi) {
  *lo = min3(min3(*lo, v.x, v.y), v.z, v.w);
  *hi = max3(max3(*hi, v.x, v.y), v.z, v.w);
}
// NaN and Inf become 0 (*bad), larger magnitudes the largest bf16.
IFQ_DEVINL void tame(float4& v, bool* bad) {
  float* f = &v.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!(fabsf(f[j]) <= 3.402823466e38f)) {
      f[j] = 0.0f;
      *bad = true;
    }
    f[j] = fminf(fmaxf(f[j], -kBf16Max), kBf16Max);
  }
}
// Whether a lane's entries need tame().
IFQ_DEVINL bool wild(float lo, float hi) { return !(lo >= -kBf16Max && hi <= kBf16Max); }

// One token's plane, 8 entries a thread.
template <int DIM>
__global__ void __launch_bounds__(kThreads) kv4_append_tokens_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LP = DIM / 8, D = 2 * DIM;
  const Kv4Arg& c = p.c;
  const int b = blockIdx.y;
  follow();
  const Kv4Seq q = kv4_seq(c, b);
  if (!q.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
    return;
  }
  const int idx = blockIdx.x * kThreads + threadIdx.x;  // below 16 x 1024 x 64
  const int part = idx % LP, plane = (idx / LP) & 3, th = idx / (4 * LP);
  const int head = th % c.kv_heads, tok = th / c.kv_heads;
  const bool live = tok < q.n_new;
  const int32_t pos = q.len - q.n_new + tok;
  uint8_t* rec = live ? kv4_record(c, b, head, pos >> 4) : nullptr;
  float4 x[2];
  const float* src = behind_wait(p.src[plane]) + (q.row0 + tok) * p.ld + head * DIM + part * 8;
  x[0] = take(src, live);
  x[1] = take(src + 4, live);
  float lo = INFINITY, hi = -INFINITY;
  widen(x[0], &lo, &hi);
  widen(x[1], &lo, &hi);
  bool bad = false;
  if (wild(lo, hi)) {
    tame(x[0], &bad);
    tame(x[1], &bad);
    lo = INFINITY, hi = -INFINITY;
    widen(x[0], &lo, &hi);
    widen(x[1], &lo, &hi);
  }
#pragma unroll
  for (int o = 1; o < LP; o *= 2) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!live) return;
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
  if (!rec) {
    if (part == 0) set_status(p.status, IFQ_DEV_RANGE);
    return;
  }
  const Group gq = group_of(lo, hi);
  const int r = pos & 15, hh = r >> 3, d = (plane & 1) * DIM + part * 8;  // d: first of the 8 stacked entries
  if (plane < 2) {
    uint32_t* w = reinterpret_cast<uint32_t*>(rec + (d >> 6) * 512 + (((r & 7) * 4 + ((d & 31) >> 3)) << 4));
    w[((d & 63) >> 5) * 2 + hh] = key_word(x[0], x[1], gq);
  } else {
    const int qb = d >> 5, g = (d & 31) >> 2, t = (r & 7) >> 1;
    uint8_t* base = rec + 8 * D + (qb >> 1) * 512 + ((qb & 1) * 2 + hh) * 4 + (r & 1) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint16_t*>(base + (((g + i) * 4 + t) << 4)) = (uint16_t)codes_of(x[i], gq);
  }
  if (part == 0) *reinterpret_cast<uint32_t*>(rec + 16 * D + (plane >> 1) * 128 + r * 8 + (plane & 1) * 4) = gq.bits;
}

// One plane of the keys (planes 0, 1) or values (2, 3) of a record of p.heads_each heads: warp w of the CTA takes plane w.
constexpr int records_ctas(int dim) { return dim == 128 ? 3 : 5; }  // that an SM holds

template <int DIM>
__global__ void __launch_bounds__(kThreads, records_ctas(DIM))
    kv4_append_records_kernel(const __grid_constant__ AppendParams p) {
  constexpr int D = 2 * DIM, CP = DIM / 32;
  static_assert(kWarps == 4, "a warp per plane");
  follow();
  const Kv4Seq seq = kv4_seq(p.c, blockIdx.z);
  if (!seq.ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
  Item it;
  if (!find_item(p, seq, blockIdx.y, blockIdx.x * p.heads_each, &it) || !it.rec) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, plane = threadIdx.x >> 5, pl = plane & 1;
  const int32_t len = it.q.len;
  auto in = [&](int r) { return it.pos0 + r >= it.first && it.pos0 + r < len; };
  const float* src = behind_wait(p.src[plane]) + (it.q.row0 + it.pos0 - it.first) * p.ld + it.head * DIM;
  const bool all = in(0) && in(15);
  bool bad = false;
  const int heads = min(p.heads_each, p.c.kv_heads - it.head);
#pragma unroll 1
  for (int head = 0; head < heads; ++head, src += DIM, it.rec += p.c.page_tiles * p.c.record_bytes) {
    if (head + 1 < heads) {  // the next head's lines on their way to L2
#pragma unroll
      for (int i = lane; i < DIM / 2; i += 32) {
        const int r = i / CP;
        if (in(r)) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + DIM + r * p.ld + i % CP * 32));
      }
    }
    uint32_t* par = reinterpret_cast<uint32_t*>(it.rec + 16 * D) + (plane >> 1) * 32 + pl;
    uint32_t words[CP][2];  // {32-column chunk of the plane, h}
    // The lanes of a group halve the groups that they share at each step of its minimum and maximum, so that a lane ends
    // with one group, makes its parameters and hands them back.
    if (plane < 2) {        // keys: tokens g + 8 h, entries 8 t .. 8 t + 7 of a chunk
      float4 v[2][CP][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < CP; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            v[h][c][i] = take(src + (g + 8 * h) * p.ld + c * 32 + t * 8 + i * 4, in(g + 8 * h));
      float lo[2], hi[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lo[h] = INFINITY, hi[h] = -INFINITY;
#pragma unroll
        for (int c = 0; c < CP; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) widen(v[h][c][i], &lo[h], &hi[h]);
        if (wild(lo[h], hi[h])) {
          lo[h] = INFINITY, hi[h] = -INFINITY;
#pragma unroll
          for (int c = 0; c < CP; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              tame(v[h][c][i], &bad);
              widen(v[h][c][i], &lo[h], &hi[h]);
            }
        }
      }
      float l, u;
      halve(lo[0], lo[1], hi[0], hi[1], 1, t & 1, &l, &u);
      both(&l, &u, 2);
      const Group own = group_of(l, u);  // of token g + 8 (t % 2)
      if (t < 2 && in(g + 8 * t)) par[(g + 8 * t) * 2] = own.bits;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Group q = group_from(own, (lane & ~3) + h);
#pragma unroll
        for (int c = 0; c < CP; ++c) words[c][h] = key_word(v[h][c][0], v[h][c][1], q);
      }
    } else {                // values: tokens 2 t + 8 h + e, entries 4 g .. 4 g + 3 of a chunk
      float4 v[2][2][CP];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int c = 0; c < CP; ++c) {
            const int r = 2 * t + 8 * h + e;
            v[h][e][c] = take(src + r * p.ld + c * 32 + g * 4, in(r));
          }
      float lo[2][2], hi[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          lo[h][e] = INFINITY, hi[h][e] = -INFINITY;
#pragma unroll
          for (int c = 0; c < CP; ++c) widen(v[h][e][c], &lo[h][e], &hi[h][e]);
          if (wild(lo[h][e], hi[h][e])) {
            lo[h][e] = INFINITY, hi[h][e] = -INFINITY;
#pragma unroll
            for (int c = 0; c < CP; ++c) {
              tame(v[h][e][c], &bad);
              widen(v[h][e][c], &lo[h][e], &hi[h][e]);
            }
          }
        }
      const int h_own = g >> 2, e_own = (g >> 1) & 1, r_own = 2 * t + 8 * h_own + e_own;
      float l2[2], u2[2], l, u;
#pragma unroll
      for (int e = 0; e < 2; ++e) halve(lo[0][e], lo[1][e], hi[0][e], hi[1][e], 16, h_own, &l2[e], &u2[e]);
      halve(l2[0], l2[1], u2[0], u2[1], 8, e_own, &l, &u);
      both(&l, &u, 4);
      const Group own = group_of(l, u);  // of token r_own
      if (!(g & 1) && in(r_own)) par[r_own * 2] = own.bits;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Group q = group_from(own, 16 * h + 8 * e + t);
#pragma unroll
          for (int c = 0; c < CP; ++c) {
            const uint32_t w = codes_of(v[h][e][c], q) << (16 * e);
            words[c][h] = e == 0 ? w : words[c][h] | w;
          }
        }
    }
#pragma unroll
    for (int c = 0; c < CP; ++c) {  // chunk ch is the words 2 (ch % 2) + h of the 16 bytes of its pair of chunks
      const int ch = pl * CP + c;
      uint8_t* dst = it.rec + (plane >> 1) * 8 * D + (ch >> 1) * 512 + lane * 16 + (ch & 1) * 8;
      if (all && CP > 1) {
        const int even = c - (CP > 1);
        if (c & 1)
          *reinterpret_cast<uint4*>(dst - 8) = make_uint4(words[even][0], words[even][1], words[c][0], words[c][1]);
      } else if (all) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(words[c][0], words[c][1]);
      } else if (plane < 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in(g + 8 * h)) reinterpret_cast<uint32_t*>(dst)[h] = words[c][h];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)  // half words: token 2 t + 8 h + (e & 1)
          if (in(2 * t + 8 * (e >> 1) + (e & 1)))
            reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(words[c][e >> 1] >> (16 * (e & 1)));
      }
    }
  }
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv4_read_records_kernel(const __grid_constant__ AppendParams p) {
  constexpr int D = 2 * DIM, CH = D / 32, CP = DIM / 32;
  follow();
  const Kv4Seq seq = kv4_seq(p.c, blockIdx.z);
  if (!seq.ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
  const int head = blockIdx.x * kWarps + (threadIdx.x >> 5);
  Item it;
  if (head >= p.c.kv_heads || !find_item(p, seq, blockIdx.y, head, &it)) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int32_t end = it.first + it.q.n_new;
  auto in = [&](int r) { return it.pos0 + r >= it.first && it.pos0 + r < end; };
  auto row = [&](float* base, int r) { return base + (it.q.row0 + it.pos0 + r - it.first) * p.ld + it.head * DIM; };
  auto put = [&](float* dst, uint32_t sm, const uint32_t (&n)[4]) {
    const float s = bf16_lo(sm), m = bf16_hi(sm);
    const float4 v = make_float4(fmaf(s, (float)n[0], m), fmaf(s, (float)n[1], m), fmaf(s, (float)n[2], m),
                                 fmaf(s, (float)n[3], m));
    __stcs(reinterpret_cast<float4*>(dst), v);
  };
  const uint32_t* par = reinterpret_cast<const uint32_t*>(it.rec + 16 * D);
  uint4 kv[2][CH / 2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int k = 0; k < CH / 2; ++k) {
      kv[x][k] = make_uint4(0, 0, 0, 0);
      if (it.rec) kv[x][k] = *reinterpret_cast<const uint4*>(it.rec + x * 8 * D + k * 512 + lane * 16);
    }
#pragma unroll
  for (int ch = 0; ch < CH; ++ch) {
    const int pl = ch / CP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4& kq = kv[0][ch / 2];
      const uint4& vq = kv[1][ch / 2];
      const uint32_t kw = ch & 1 ? (h ? kq.w : kq.z) : (h ? kq.y : kq.x);
      const uint32_t vw = ch & 1 ? (h ? vq.w : vq.z) : (h ? vq.y : vq.x);
      const int rk = g + 8 * h;
      if (in(rk)) {
        const uint32_t sm = it.rec ? par[rk * 2 + pl] : 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t n[4] = {(kw >> (8 * i)) & 15u, (kw >> (16 + 8 * i)) & 15u, (kw >> (4 + 8 * i)) & 15u,
                                 (kw >> (20 + 8 * i)) & 15u};
          put(row(p.dst[pl], rk) + (ch % CP) * 32 + t * 8 + i * 4, sm, n);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rv = 2 * t + 8 * h + e;
        if (!in(rv)) continue;
        const uint32_t sm = it.rec ? par[32 + rv * 2 + pl] : 0u, w = vw >> (16 * e);
        const uint32_t n[4] = {w & 15u, (w >> 4) & 15u, (w >> 8) & 15u, (w >> 12) & 15u};
        put(row(p.dst[2 + pl], rv) + (ch % CP) * 32 + g * 4, sm, n);
      }
    }
  }
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv4_read_tokens_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LP = DIM / 8, D = 2 * DIM;
  const Kv4Arg& c = p.c;
  const int b = blockIdx.y;
  follow();
  const Kv4Seq q = kv4_seq(c, b);
  if (!q.ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
  const int idx = blockIdx.x * kThreads + threadIdx.x;
  const int part = idx % LP, plane = (idx / LP) & 3, th = idx / (4 * LP);
  const int head = th % c.kv_heads, tok = th / c.kv_heads;
  if (tok >= q.n_new) return;
  float o[8] = {};
  uint8_t* rec = nullptr;
  const int32_t pos = q.len - q.n_new + tok;
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
  const bool tokens = p.c.n_new < 16;
  if (tokens) {  // threads of 8 entries
    const int64_t blocks = ((int64_t)p.c.n_new * p.c.kv_heads * (DIM / 2) + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)blocks, (unsigned)p.c.B);
    auto kernel = read ? kv4_read_tokens_kernel<DIM> : kv4_append_tokens_kernel<DIM>;
    return launch_following<AppendParams>(kernel, grid, kThreads, 0, 1, p, s);
  } else {       // the records that n_new tokens can touch, a CTA (appending) or a warp each; heads fastest, so that
                 // CTAs that run together read neighbouring columns
    const unsigned tiles = (unsigned)(((int64_t)p.c.n_new + 14) / 16 + 1);
    const unsigned heads = (unsigned)p.c.kv_heads;
    auto kernel = read ? kv4_read_records_kernel<DIM> : kv4_append_records_kernel<DIM>;
    AppendParams pp = p;
    // up to 8 heads, as long as the GPU's places are taken twice (2900 tokens of 32 heads 22.2 us, with 1 head 27.3;
    // with 16, which take them once, 34)
    pp.heads_each = 8;
    while (pp.heads_each > 1 && (int64_t)p.c.B * tiles * ((heads + pp.heads_each - 1) / pp.heads_each) <
                                    2 * 148 * records_ctas(DIM))
      pp.heads_each /= 2;
    const unsigned each = read ? kWarps : (unsigned)pp.heads_each;
    return launch_following<AppendParams>(kernel, dim3((heads + each - 1) / each, tiles, (unsigned)p.c.B), kThreads, 0,
                                          1, pp, s);
  }
}

cudaError_t dispatch(const ifq_kv4_cache& c, const AppendParams& p, bool read, cudaStream_t s) {
  if (c.dim == 32) return launch<32>(p, read, s);
  if (c.dim == 64) return launch<64>(p, read, s);
  return launch<128>(p, read, s);
}

}  // namespace

cudaError_t launch_kv4_append(const ifq_kv4_cache& c, const float* k_re, const float* k_im, const float* v_re,
                              const float* v_im, int64_t ld, uint32_t* dev_status, cudaStream_t s) {
  AppendParams p = {kv4_arg(c), {k_re, k_im, v_re, v_im}, {}, ld, 1, dev_status};
  return dispatch(c, p, false, s);
}

cudaError_t launch_kv4_read(const ifq_kv4_cache& c, float* k_re, float* k_im, float* v_re, float* v_im, int64_t ld,
                            uint32_t* dev_status, cudaStream_t s) {
  AppendParams p = {kv4_arg(c), {}, {k_re, k_im, v_re, v_im}, ld, 1, dev_status};
  return dispatch(c, p, true, s);
}

}  // namespace ifq

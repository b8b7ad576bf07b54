// Decode attention over the 4-bit key/value cache: for each query head of each new token
//   score_j = scale (q_re . k_re,j + q_im . k_im,j),  o = sum_j softmax(score)_j v_j,
// keys j <= the token's position, o's planes summed separately.
//
// One pass over the cache with the running maximum and sum of the softmax.  A warp takes 32 keys at a
// time (two records, copied asynchronously into a ring of its own): keys are the rows of the matrix
// instruction's A operand, queries the columns of B, all in fp16 with float32 sums.
//   codes  four bits of a word under a mask are already a number: n 2^-24 in bits 0-3 of an fp16, 16 n 2^-24 in
//          bits 4-7 (subnormal and first normal numbers share one spacing), so an operand register
//          costs one AND; the 16 is undone in q's columns (keys) or in the output's rows (values)
//   q      float32 times scale log2 e, scaled by a power of two per row to below 2^15 and split into two fp16
//          terms (2^-22 of the row's largest entry): two neighbouring columns where a tile has up to 4
//          query rows, two products into the same sums where it has 8
//   K      score = scale sum_planes s (codes . q) + m sum(q), s and m of a key's plane, in float32
//   P      p = 2^(score - ref), ref the maximum when it was last raised: it is raised, and all sums rescaled,
//          only when a score passes it by more than 2^kSlack, so that rescaling stays rare;
//          p s 2^(15 - kSlack) / cap as one fp16 term (2^-11 relative), cap a power of two above every s
//          seen (raised the same way), transposed in registers (movmatrix) from the score layout
//          into the B operand; o = sum_j (p s)_j codes_j + sum_j p_j m_j, the second sum in float32
// A lane holds the scores of one query row (of two, in tiles of 8) for the keys g and g + 8 of a record.
//
// Work split.  A pair is a key/value head and a tile of 4 or 8 query rows of a sequence; its work is its
// units of 32 keys.  The four warps of a CTA share a run of units and join their parts in shared memory.
//   few units   a cluster of up to 8 CTAs per pair, joined through distributed shared memory: one launch (777 tokens
//               of 32 heads 6.4 us, against 11.4 us by the other form; 9 sequences of up to 3001 tokens, 5 heads,
//               4 new tokens 10.6 us against 13.7)
//   otherwise   one CTA per place on the GPU, each with an equal run of the units of all pairs in a row (counted
//               on the device, where the lengths are): a CTA ends one pair, does whole ones, begins another; the
//               pairs that a CTA's end cuts are joined by a second, small kernel.  However ragged the
//               lengths, all CTAs end together (8 ragged sequences of up to 33 thousand tokens 41 us; cut into 4
//               parts each 79 us).
// All joins add in a fixed order.
//
// Every pair is a pass of its own over its head's records: query rows beyond 8 (new tokens times shared heads) cost
// another pass each 8 (8 sequences of 20000 tokens, 8 heads, 8 query heads each: 1 new token 47 us, 4 148 us, 16 542 us).
//
// The form is chosen on the host by the positions that the page table has room for, not by the lengths, which are on the
// device: 777 tokens of 32 heads in a table of 131072 positions take the counted form.
//
// Rounding: the weights enter the second product as one fp16 term.  The output is bf16, whose rounding is 8 times
// coarser; with a second term the error against 64 bits goes from 1.73 to 1.72 10^-3 (131072 tokens) and the time from 50.0
// to 51.8 us, for 32 ragged sequences from 74.7 to 80.9 us (L2 flushed).  q needs two: the absolute error of a score is
// the relative one of its weight, and scores are large.
//
// Bound: 131072 tokens of 8 heads (64 query heads, 151 MB) take 41 us (captured, caches that L2 does not hold).  About 14
// us of that do not grow with the length: two launches, counting, a pair's q and first copies, the joins.  Each further
// 131072 tokens take 27 us, 87 % of the copy rate: 288 warp instructions per record and pair of 8 rows (80 to unmask codes,
// 24 matrix instructions, 60 for scores and weights), issued at 60 % of the slots.  In all it is bound by latency: 11 warps
// an SM, whose chains of products, scores and weights keep issue at 48 % and no pipe above 44 %.  The registers spilled for
// 8 rows at dim 64 are read 6 times a warp, outside the loop over the records.
#include "ifq_internal.h"
#include "kv4_common.cuh"

#include <cuda_fp16.h>

namespace ifq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;                  // keys of a warp's step: two records
constexpr int kStages = 2;
constexpr int kSlack = 6;                  // how far (log2) a score may pass the reference
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSeqs = 8 * kThreads;     // sequences that a CTA counts, up to 8 a thread

// CTAs that an SM holds (its registers decide).
__host__ __device__ constexpr int ctas_per_sm(int dim, int nt) { return dim == 128 ? 2 : dim == 64 && nt == 2 ? 3 : 4; }

struct AttnParams {
  Kv4Arg c;
  const float* q[2];
  uint16_t* o[2];
  int64_t ldq, ldo;
  float scale2;      // scale log2 e
  int32_t shared;    // query heads of a key/value head
  int32_t cluster, qtiles;
  int32_t counted;   // equal runs of the units of all pairs (else a cluster per pair)
  int32_t by_pair;   // a Cut for every pair, else one for every CTA
  float* ws_o;       // [CTAs][2][QR][D]: partial results of the pair that a CTA ends, and of the one that it begins
  float2* ws_ml;     // [CTAs][2][QR]: maximum (log2), sum
  struct Cut* ws_cut;  // [CTAs], of which [pairs] are used where there are fewer
  uint32_t* status;
};

// What CTAs first .. last did of a pair is joined.  pair < 0: nothing (a pair that one CTA had whole, or a CTA that
// left no pair begun).  Read 16 bytes at a time.
struct alignas(16) Cut {
  int32_t pair, first, last, n_new;
  int64_t row0;
};

IFQ_DEVINL float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 x 8 transpose of 16-bit elements over a warp.
IFQ_DEVINL uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

IFQ_DEVINL uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

IFQ_DEVINL void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
IFQ_DEVINL void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The four operand registers of a word: codes times 2^-24 (first and third) and 2^-20 (second and fourth).
IFQ_DEVINL void codes_f16(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t v = w >> 8;
  a[0] = w & 0x000F000Fu;
  a[1] = w & 0x00F000F0u;
  a[2] = v & 0x000F000Fu;
  a[3] = v & 0x00F000F0u;
}

// 2^e as a float, for -126 <= e <= 127.
IFQ_DEVINL float pow2(int e) { return __int_as_float((e + 127) << 23); }

IFQ_DEVINL int32_t units_of(int32_t len) { return (len + kUnit - 1) / kUnit; }

// A CTA's run of units of one pair.
struct Segment {
  Kv4Seq seq;
  int32_t b, pair, begin, end, units;  // units: all of the pair; at least one, which writes an empty row's zeros
};

// Starting a pair (its q, the first copies, the joins) costs a CTA about as much as this many units: counted runs
// weigh a pair as its units and kStart more, those first.  (With 6, 64 ragged sequences of 8 heads take 93 us, with
// 16 to 32 65 us; equal lengths hardly change.)
constexpr int kStart = 24;

IFQ_DEVINL float2 ld_cluster2(const void* smem, uint32_t rank) {
  uint32_t a;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

template <int DIM, int NT>
struct Layout {
  static constexpr int D = 2 * DIM, CH = D / 32, QR = 4 * NT;
  static constexpr int kRecord = 16 * D + 256;
  static constexpr int kStage = 2 * kRecord;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = NT * CH * 512;                     // B operands of q: [term or 0][chunk][lane]
  static constexpr int kBytes = kRing + kQ;
  static constexpr int kSums = kWarps * QR * D * 4;            // in the ring's memory
  static_assert(kSums <= kRing, "the sums reuse the ring");
};

template <int DIM, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(DIM, NT))
    kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  using Y = Layout<DIM, NT>;
  constexpr int D = Y::D, CH = Y::CH, CP = DIM / 32, QR = Y::QR, T4 = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float qsum[QR][2];             // 2^-24 sum of a scaled query's plane
  __shared__ int qexp[QR];                  // exponent of a query row's largest entry
  __shared__ float2 mls[kWarps][QR];
  __shared__ float2 ml_cta[QR];
  uint4* qs = reinterpret_cast<uint4*>(smem + Y::kRing);
  const Kv4Arg& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = (int)blockIdx.x % p.cluster;
  follow();

  // The runs.  Thread i counts the sequences i per_thread .. + per_thread - 1.
  __shared__ unsigned long long warp_sums[kWarps];
  __shared__ unsigned long long counts[kThreads][2];  // a thread's own: the weight before its sequences, and theirs
  __shared__ Segment found;
  __shared__ int32_t step;  // its weight
  auto weight = [&](const Kv4Seq& q) -> unsigned long long {
    return (unsigned long long)(max(1, units_of(q.len)) + kStart) * ((q.n_new * p.shared + QR - 1) / QR * c.kv_heads);
  };
  const int per_thread = (c.B + kThreads - 1) / kThreads;
  __shared__ unsigned long long runs[3];                // begin of what is left, end, length of a run
  if (p.counted) {
    unsigned long long own = 0;
    for (int i = 0; i < per_thread; ++i) {
      const int b = threadIdx.x * per_thread + i;
      if (b >= c.B) break;
      const Kv4Seq q = kv4_seq(c, b);
      if (!q.ok && blockIdx.x == 0) set_status(p.status, IFQ_DEV_RANGE);
      own += weight(q);
    }
    unsigned long long sum = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned long long up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    unsigned long long total = 0, before = sum - own;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    counts[threadIdx.x][0] = before;
    counts[threadIdx.x][1] = own;
    if (threadIdx.x == 0) {
      const unsigned long long run = max((total + gridDim.x - 1) / gridDim.x, (unsigned long long)(kStart + kWarps));
      runs[0] = min(total, blockIdx.x * run);
      runs[1] = min(total, runs[0] + run);
      runs[2] = run;
      if (!p.by_pair) p.ws_cut[blockIdx.x].pair = -1;
    }
    __syncthreads();
  }

  for (;;) {
    if (p.counted) {
      // the thread whose sequences hold the begin
      const unsigned long long at = runs[0], end = runs[1], run = runs[2];
      if (at >= end) return;
      const unsigned long long before = counts[threadIdx.x][0];
      if (at >= before && at - before < counts[threadIdx.x][1]) {
        unsigned long long u = at - before;
        for (int i = 0; i < per_thread; ++i) {
          const int b = threadIdx.x * per_thread + i;
          const Kv4Seq q = kv4_seq(c, b);
          const unsigned long long all = weight(q);
          if (u < all) {
            const int32_t units = max(1, units_of(q.len)), whole = units + kStart;
            const int32_t pair = (int32_t)(u / whole), from = (int32_t)(u - (unsigned long long)pair * whole);
            const int32_t to = end - at < whole - from ? from + (int32_t)(end - at) : whole;
            found = {q, b, pair, max(0, from - kStart), max(0, to - kStart), units};
            const unsigned long long start = at - from + kStart;  // of the pair's first unit
            if (found.begin == 0 && found.end > 0 && (found.end < units || p.by_pair))  // begun here
              p.ws_cut[p.by_pair ? b * (c.kv_heads * p.qtiles) + pair : (int)blockIdx.x] = {
                  found.end < units ? pair : -1, (int)blockIdx.x, (int)((start + units - 1) / run), q.n_new, q.row0};
            step = to - from;
            break;
          }
          u -= all;
        }
      }
    } else if (threadIdx.x == 0) {
      const Kv4Seq q = kv4_seq(c, blockIdx.z);
      if (!q.ok && blockIdx.x == 0 && blockIdx.y == 0) set_status(p.status, IFQ_DEV_RANGE);
      const int32_t units = max(1, units_of(q.len)), per = (units + p.cluster - 1) / p.cluster;
      const int32_t qtiles = (q.n_new * p.shared + QR - 1) / QR;
      // (pairs past the sequence's own have no rows and are left out below, by the whole cluster)
      found = {q, (int)blockIdx.z, (int)blockIdx.y < qtiles * c.kv_heads ? (int)blockIdx.y : -1, min(units, rank * per),
               min(units, (rank + 1) * per), units};
    }
    __syncthreads();
    if (found.pair < 0) return;
    if (p.counted && threadIdx.x == 0) runs[0] += step;
    if (p.counted && found.begin == found.end) {  // a run that ends before the pair's first unit
      __syncthreads();
      continue;
    }
    const int b = found.b;
    const Kv4Seq sq = found.seq;
    const int qtiles = (sq.n_new * p.shared + QR - 1) / QR;
    const int kvh = found.pair / qtiles, qt = found.pair % qtiles;
    const int nrows = sq.n_new * p.shared - qt * QR;  // query rows of this tile

    // this warp's tiles (records) of the sequence, contiguous
    const int32_t per = (found.end - found.begin + kWarps - 1) / kWarps;
    const int32_t tiles = min((sq.len + 15) >> 4, found.end * 2);
    const int32_t t_begin = min(tiles, (found.begin + warp * per) * 2);
    const int32_t t_end = min(tiles, t_begin + per * 2);

    // Record numbers, 32 tiles at a time (lane l: tile base + l), the next 32 on their way.
    auto fetch = [&](int32_t base) -> uint32_t {
      const int32_t tl = base + lane;
      if (tl >= t_end) return 0xFFFFFFFFu;
      const int32_t pc = (int32_t)((uint32_t)tl / (uint32_t)c.page_tiles), in = tl - pc * c.page_tiles;
      const int32_t page = ld_after(c.page_table + (int64_t)b * c.table_cols + pc);
      if (page < 0 || page >= c.pages) {
        set_status(p.status, IFQ_DEV_RANGE);
        return 0xFFFFFFFFu;
      }
      return ((uint32_t)page * c.kv_heads + kvh) * c.page_tiles + in;
    };
    uint32_t rec_now = fetch(t_begin), rec_next = fetch(t_begin + 32);
    const uint32_t ring = smem_u32(smem) + warp * kStages * Y::kStage + lane * 16;
    const bool even_pages = (c.page_tiles & 1) == 0;  // the two records of a step are neighbours in a page
    uint32_t ok = 0;          // bit 2 slot + i: record i of the slot's stage is there
    int32_t tl = t_begin;     // first tile of the next load
    auto load = [&](int slot) {
      if (tl < t_end) {
        ok &= ~(3u << (2 * slot));
        if (even_pages && tl + 1 < t_end) {
          const uint32_t r = __shfl_sync(0xffffffffu, rec_now, (tl - t_begin) & 31);
          if (r != 0xFFFFFFFFu) {
            ok |= 3u << (2 * slot);
            const uint8_t* src = c.records + (uint64_t)r * Y::kRecord + lane * 16;
            const uint32_t dst = ring + slot * Y::kStage;
#pragma unroll
            for (int v = 0; v < Y::kStage / 512; ++v) cp_async16(dst + v * 512, src + v * 512);
          }
        } else
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t r = __shfl_sync(0xffffffffu, rec_now, (tl - t_begin + i) & 31);
          if (r != 0xFFFFFFFFu) {
            ok |= 1u << (2 * slot + i);
            const uint8_t* src = c.records + (uint64_t)r * Y::kRecord + lane * 16;
            const uint32_t dst = ring + slot * Y::kStage + i * Y::kRecord;
#pragma unroll
            for (int v = 0; v < Y::kRecord / 512; ++v) cp_async16(dst + v * 512, src + v * 512);
            if (lane < Y::kRecord % 512 / 16) cp_async16(dst + Y::kRecord / 512 * 512, src + Y::kRecord / 512 * 512);
          }
        }
        tl += 2;
        if (((tl - t_begin) & 31) == 0) {
          rec_now = rec_next;
          rec_next = fetch(tl + 32);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) load(st);

    // q, a warp per row: lane l has the entries E l .. E l + E - 1.  The row's exponent, its plane sums, and its two
    // fp16 terms at their places in the operands.
    constexpr int E = D / 32;
    for (int row = warp; row < QR; row += kWarps) {
      float v[E] = {};
      if (row < nrows) {
        const int rr = qt * QR + row, tok = rr / p.shared, head = kvh * p.shared + rr % p.shared;
        const float* src = p.q[lane / 16] + (sq.row0 + tok) * p.ldq + head * DIM + lane % 16 * E;
#pragma unroll
        for (int j = 0; j < E; j += 2) {
          const float2 x = ld_after(reinterpret_cast<const float2*>(src + j));
          v[j] = x.x;
          v[j + 1] = x.y;
        }
      }
      float mx = 0.0f, sum = 0.0f;
      bool bad = false;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        v[j] *= p.scale2;
        bad |= !(fabsf(v[j]) <= 3.402823466e38f);  // q or the scale
        mx = fmaxf(mx, fabsf(v[j]));
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (mx > 0x1p99f * kLog2e) {  // |scale q| above 2^99, whose scores could overflow: the row counts as not finite
        bad = true;
        v[0] = NAN;
      }
      if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
      // mx < 2^(e + 1); a zero or tiny row keeps the smallest exponent
      const int e = max((__float_as_int(mx) >> 23) - 127, -100);
      const float f = pow2(14 - e);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        v[j] *= f;
        sum += v[j];
        if ((lane * E + j) & 2) v[j] *= 0x1p-4f;  // entries 2, 3, 6, 7 of a word meet codes times 16
      }
#pragma unroll
      for (int o = 8; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) qexp[row] = e;
      if (lane % 16 == 0) qsum[row][lane / 16] = sum * 0x1p-24f;
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        const int d = lane * E + j, ch = d >> 5, tt = (d & 31) >> 3;
        const uint32_t hi = pack_f16(v[j], v[j + 1]);
        const __half2 h2 = *reinterpret_cast<const __half2*>(&hi);
        const uint32_t lo = pack_f16(v[j] - __low2float(h2), v[j + 1] - __high2float(h2));
        // term p of row r: column 2 r + p of the one n tile, or column r of tile p
        uint32_t* q0 = reinterpret_cast<uint32_t*>(qs + ch * 32 + (NT == 1 ? 8 * row : 4 * row) + tt) + ((d & 7) >> 1);
        q0[0] = hi;
        q0[NT == 1 ? 16 : CH * 128] = lo;
      }
    }
    __syncthreads();

    // This lane's query rows: t, or 2 t and 2 t + 1.
    float qs2[NT][2], cs[NT];
    int32_t visible[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = NT * t + j;
      qs2[j][0] = qsum[row][0];
      qs2[j][1] = qsum[row][1];
      cs[j] = pow2(min(qexp[row], 100) + 10);  // undoes the 2^-24 of the codes and the row's 2^(14 - e)
      visible[j] = row < nrows ? sq.len - sq.n_new + (qt * QR + row) / p.shared + 1 : 0;
    }
    // keys below this are seen by every row of the tile (rows past the last count as seeing all)
    const int32_t vis_all = sq.len - sq.n_new + qt * QR / p.shared + 1;

    float acc[CH][2][4];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
    float m_run[NT], l_run[NT], pm[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_run[nt] = -INFINITY;
      l_run[nt] = pm[nt][0] = pm[nt][1] = 0.0f;
    }
    float cap[2] = {0.0f, 0.0f}, to_w[2] = {0.0f, 0.0f};  // per plane: the cap on s, 2^(15 - kSlack) / cap

    const uint8_t* stage0 = smem + warp * kStages * Y::kStage;
    auto unit = [&](int slot, int32_t key0) {
      const uint8_t* base = stage0 + slot * Y::kStage;
      const bool full = key0 + kUnit <= vis_all && ((ok >> (2 * slot)) & 3u) == 3u;
      // scores in units of 1 / cs: {record, row, key g or g + 8}
      float sc[2][NT][2];
      float s4[2][2][4];  // {record, plane}
#pragma unroll
      for (int v = 0; v < T4; ++v) {
        uint4 w4[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w4[i] = *reinterpret_cast<const uint4*>(base + i * Y::kRecord + v * 512 + lane * 16);
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int ch = 2 * v + cc, pl = ch / CP;
          uint4 bq[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) bq[j] = qs[(j * CH + ch) * 32 + lane];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t lo[4], hi[4];
            codes_f16(cc ? w4[i].z : w4[i].x, lo);
            codes_f16(cc ? w4[i].w : w4[i].y, hi);
            if (ch % CP == 0) mma_f16_first(s4[i][pl], lo[0], hi[0], lo[1], hi[1], bq[0].x, bq[0].y);
            else mma_f16(s4[i][pl], lo[0], hi[0], lo[1], hi[1], bq[0].x, bq[0].y);
            mma_f16(s4[i][pl], lo[2], hi[2], lo[3], hi[3], bq[0].z, bq[0].w);
            if (NT == 2) {
              mma_f16(s4[i][pl], lo[0], hi[0], lo[1], hi[1], bq[NT - 1].x, bq[NT - 1].y);
              mma_f16(s4[i][pl], lo[2], hi[2], lo[3], hi[3], bq[NT - 1].z, bq[NT - 1].w);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 par = *reinterpret_cast<const uint2*>(base + i * Y::kRecord + 16 * D + (g + 8 * h) * 8);
          const float k0 = bf16_lo(par.x), m0 = bf16_hi(par.x), k1 = bf16_lo(par.y), m1 = bf16_hi(par.y);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float a0 = NT == 1 ? s4[i][0][2 * h] + s4[i][0][2 * h + 1] : s4[i][0][2 * h + j];
            const float a1 = NT == 1 ? s4[i][1][2 * h] + s4[i][1][2 * h + 1] : s4[i][1][2 * h + j];
            sc[i][j][h] = fmaf(k0, a0, fmaf(k1, a1, fmaf(m0, qs2[j][0], m1 * qs2[j][1])));
          }
        }
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (key0 + 16 * i + g + 8 * h >= visible[nt] || !((ok >> (2 * slot + i)) & 1u)) sc[i][nt][h] = -INFINITY;
      }
      float mn[NT];  // this lane's largest score of a row
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mn[nt] = cs[nt] * fmaxf(fmaxf(sc[0][nt][0], sc[0][nt][1]), fmaxf(sc[1][nt][0], sc[1][nt][1]));
        grew |= mn[nt] > m_run[nt] + kSlack;
      }
      // the values' scales and minima of this lane's keys: {record, key, plane}; 0 for keys that do not exist
      float vs[2][2][2], vm[2][2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint2 par = *reinterpret_cast<const uint2*>(base + i * Y::kRecord + 16 * D + 128 + (g + 8 * h) * 8);
          if (!full && (key0 + 16 * i + g + 8 * h >= sq.len || !((ok >> (2 * slot + i)) & 1u))) par = make_uint2(0, 0);
          vs[i][h][0] = bf16_lo(par.x);
          vm[i][h][0] = bf16_hi(par.x);
          vs[i][h][1] = bf16_lo(par.y);
          vm[i][h][1] = bf16_hi(par.y);
        }
      float top[2];
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
        top[pl] = fmaxf(fmaxf(vs[0][0][pl], vs[0][1][pl]), fmaxf(vs[1][0][pl], vs[1][1][pl]));
      grew |= top[0] > cap[0] || top[1] > cap[1];
      if (__any_sync(0xffffffffu, grew)) {
        float f[2];  // what a raised cap does to a plane's sums
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
          float mx = top[pl];
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          f[pl] = 1.0f;
          if (mx > cap[pl]) {
            // mx < 2^(e - 1): room to grow.  From 2^-118 up, so that to_w is a float32: a weight is then off by 2^-34
            // of cap or, for smaller scales, 2^-152, which is nothing next to float32's own last step
            const int e = min(max((__float_as_int(mx) >> 23) - 127 + 2, -118), 126);
            f[pl] = cap[pl] * pow2(-e);
            cap[pl] = pow2(e);
            to_w[pl] = pow2(15 - kSlack - e);
          }
        }
        float al[2] = {1.0f, 1.0f};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int o = 4; o < 32; o *= 2) mn[nt] = fmaxf(mn[nt], __shfl_xor_sync(0xffffffffu, mn[nt], o));
          mn[nt] = fmaxf(mn[nt], m_run[nt]);
          al[nt] = mn[nt] == -INFINITY ? 1.0f : ex2(m_run[nt] - mn[nt]);
          m_run[nt] = mn[nt];
          l_run[nt] *= al[nt];
          pm[nt][0] *= al[nt];
          pm[nt][1] *= al[nt];
        }
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[ch][j][e] *= al[e & 1] * f[ch / CP];
      }
      float mb[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mb[nt] = m_run[nt] == -INFINITY ? 0.0f : m_run[nt];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t pb[2][2];  // B operands of p s: plane, keys 0-7 / 8-15
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w0 = vs[i][h][0] * to_w[0], w1 = vs[i][h][1] * to_w[1];
          float pr[2] = {0.0f, 0.0f};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            pr[nt] = ex2(fmaf(sc[i][nt][h], cs[nt], -mb[nt]));
            l_run[nt] += pr[nt];
            pm[nt][0] = fmaf(pr[nt], vm[i][h][0], pm[nt][0]);
            pm[nt][1] = fmaf(pr[nt], vm[i][h][1], pm[nt][1]);
          }
          pb[0][h] = movmatrix(pack_f16(pr[0] * w0, pr[1] * w0));
          pb[1][h] = movmatrix(pack_f16(pr[0] * w1, pr[1] * w1));
        }
#pragma unroll
        for (int v = 0; v < T4; ++v) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(base + i * Y::kRecord + 8 * D + v * 512 + lane * 16);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int ch = 2 * v + cc, pl = ch / CP;
            uint32_t lo[4], hi[4];
            codes_f16(cc ? w4.z : w4.x, lo);
            codes_f16(cc ? w4.w : w4.y, hi);
            mma_f16(acc[ch][0], lo[0], lo[1], hi[0], hi[1], pb[pl][0], pb[pl][1]);
            mma_f16(acc[ch][1], lo[2], lo[3], hi[2], hi[3], pb[pl][0], pb[pl][1]);
          }
        }
      }
    };

    for (int32_t tt = t_begin; tt < t_end;) {
#pragma unroll
      for (int slot = 0; slot < kStages; ++slot, tt += 2) {
        if (tt >= t_end) break;
        cp_async_wait<kStages - 2>();
        __syncwarp();  // every lane's copies of the stage are in, and the previous stage has been read
        load((slot + kStages - 1) % kStages);
        unit(slot, tt * 16);
      }
    }
    cp_async_wait<0>();
    __syncthreads();

    // the warps' parts, then their sum, then the cluster's
    float* os = reinterpret_cast<float*>(smem);  // [warp][row][D]
    // undo the codes' 2^-24 (2^-20 in the second half of the instruction's rows) and the weights' scaling
    constexpr float kLow = (float)(1 << (9 + kSlack)), kHigh = (float)(1 << (5 + kSlack));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) {
        l_run[nt] += __shfl_xor_sync(0xffffffffu, l_run[nt], o);
        pm[nt][0] += __shfl_xor_sync(0xffffffffu, pm[nt][0], o);
        pm[nt][1] += __shfl_xor_sync(0xffffffffu, pm[nt][1], o);
      }
      const int row = NT * t + nt;
      if (g == 0) mls[warp][row] = make_float2(m_run[nt], l_run[nt]);
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        const float pmv = pm[nt][ch / CP], k = cap[ch / CP];
        float4 v;
        v.x = fmaf(acc[ch][0][nt] * kLow, k, pmv);
        v.y = fmaf(acc[ch][0][2 + nt] * kHigh, k, pmv);
        v.z = fmaf(acc[ch][1][nt] * kLow, k, pmv);
        v.w = fmaf(acc[ch][1][2 + nt] * kHigh, k, pmv);
        *reinterpret_cast<float4*>(&os[(warp * QR + row) * D + ch * 32 + 4 * g]) = v;
      }
    }
    __syncthreads();
    const bool joined = p.cluster > 1;
    const bool whole = joined || (found.begin == 0 && found.end == found.units);
    // o and (M, l) of a row's pair of entries: to the output, or as a partial result
    auto store = [&](int row, int d, float M, float l, float o0, float o1) {
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int rr = qt * QR + row, tok = rr / p.shared, head = kvh * p.shared + rr % p.shared;
        *reinterpret_cast<uint32_t*>(p.o[d / DIM] + (sq.row0 + tok) * p.ldo + head * DIM + d % DIM) =
            pack_bf16(o0 * inv, o1 * inv);
      } else {
        const int64_t place = ((int64_t)blockIdx.x * 2 + (found.begin == 0)) * QR + row;
        *reinterpret_cast<float2*>(p.ws_o + place * D + d) = make_float2(o0, o1);
        if (d == 0) p.ws_ml[place] = make_float2(M, l);
      }
    };
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
        const float2 v = *reinterpret_cast<const float2*>(&os[(w * QR + row) * D + d]);
        l += f * mls[w][row].y;
        o0 += f * v.x;
        o1 += f * v.y;
      }
      if (joined) {
        // over warp 0's part, which this thread alone has read
        *reinterpret_cast<float2*>(&os[row * D + d]) = make_float2(o0, o1);
        if (d == 0) ml_cta[row] = make_float2(M, l);
      } else {
        store(row, d, M, l, o0, o1);
      }
    }
    if (!joined) {
      if (!p.counted) return;
      __syncthreads();  // the sums have been read: the next run's copies may overwrite them
      continue;
    }
    cluster_sync();
    const int pairs = QR * (D / 2) / p.cluster;
    for (int i = rank * pairs + threadIdx.x; i < (rank + 1) * pairs; i += kThreads) {
      const int row = i / (D / 2), d = (i % (D / 2)) * 2;
      if (row >= nrows) break;
      float M = -INFINITY;
      for (int k = 0; k < p.cluster; ++k) M = fmaxf(M, ld_cluster2(&ml_cta[row], k).x);
      const float ms = M == -INFINITY ? 0.0f : M;
      float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
      for (int k = 0; k < p.cluster; ++k) {
        const float2 ml = ld_cluster2(&ml_cta[row], k), v = ld_cluster2(&os[row * D + d], k);
        const float f = ex2(ml.x - ms);
        l += f * ml.y;
        o0 += f * v.x;
        o1 += f * v.y;
      }
      store(row, d, M, l, o0, o1);
    }
    cluster_sync();  // no CTA leaves while its sums are being read
    return;
  }
}

// The parts of the pairs that CTAs' ends cut, added in a fixed order.  CTA (i, row): a row of pair i, or of the pair
// that CTA i of the main kernel left begun, whichever are fewer (blocks with nothing to do cost: 8 pairs in 444 CTAs
// 45.2 us, as 8 blocks a row 41.3).  Its warps take the parts in turn, four at a time in flight (a pair of 131072 keys has 56).
template <int DIM, int W>
__global__ void __launch_bounds__(W * 32) kv4_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int D = 2 * DIM, V = D / 64;
  __shared__ float os[W][D];
  __shared__ float2 mls[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, qr = gridDim.y, row = blockIdx.y;
  follow();  // the main kernel's results
  const int4 cut = ld_after(reinterpret_cast<const int4*>(p.ws_cut + blockIdx.x));  // pair, first, last, n_new
  if (p.by_pair) {  // pairs that a sequence does not have are not written
    const int of_seq = p.c.kv_heads * p.qtiles;
    const Kv4Seq q = kv4_seq(p.c, (int)blockIdx.x / of_seq);
    if ((int)blockIdx.x % of_seq >= (q.n_new * p.shared + qr - 1) / qr * p.c.kv_heads) return;
  }
  if (cut.x < 0) return;
  const int64_t row0 = ld_after(&p.ws_cut[blockIdx.x].row0);
  const int rows = cut.w * p.shared, qtiles = (rows + qr - 1) / qr;
  const int kvh = cut.x / qtiles, rr = cut.x % qtiles * qr + row;
  if (rr >= rows) return;
  // part s: what CTA first + s did of the pair; the first began it, the others found it begun
  const int parts = cut.z - cut.y + 1;
  auto place = [&](int s) { return ((int64_t)(cut.y + s) * 2 + (s == 0)) * qr + row; };
  float M = -INFINITY, l = 0.0f;
  float2 o[V] = {};
  for (int s0 = warp; s0 < parts; s0 += 4 * W) {
    float2 ml[4], v[4][V];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k * W;
      ml[k] = make_float2(-INFINITY, 0.0f);
      if (s < parts) ml[k] = ld_after(p.ws_ml + place(s));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[k][i] = make_float2(0.0f, 0.0f);
        if (s < parts) v[k][i] = ld_after(reinterpret_cast<const float2*>(p.ws_o + place(s) * D + i * 64 + lane * 2));
      }
    }
    const float top = fmaxf(fmaxf(fmaxf(M, ml[0].x), fmaxf(ml[1].x, ml[2].x)), ml[3].x);
    const float ms = top == -INFINITY ? 0.0f : top, f0 = ex2(M - ms);
    M = top;
    l *= f0;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i].x *= f0, o[i].y *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = ex2(ml[k].x - ms);
      l = fmaf(f, ml[k].y, l);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i].x = fmaf(f, v[k][i].x, o[i].x);
        o[i].y = fmaf(f, v[k][i].y, o[i].y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) *reinterpret_cast<float2*>(&os[warp][i * 64 + lane * 2]) = o[i];
  if (lane == 0) mls[warp] = make_float2(M, l);
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  const int d = threadIdx.x * 2;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) M = fmaxf(M, mls[w].x);
  const float ms = M == -INFINITY ? 0.0f : M;
  float o0 = 0.0f, o1 = 0.0f;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float f = ex2(mls[w].x - ms);
    const float2 v = *reinterpret_cast<const float2*>(&os[w][d]);
    l = fmaf(f, mls[w].y, l);
    o0 = fmaf(f, v.x, o0);
    o1 = fmaf(f, v.y, o1);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = rr / p.shared, head = kvh * p.shared + rr % p.shared;
  *reinterpret_cast<uint32_t*>(p.o[d / DIM] + (row0 + tok) * p.ldo + head * DIM + d % DIM) =
      pack_bf16(o0 * inv, o1 * inv);
}

struct Plan {
  int nt, qtiles, cluster, ctas;  // ctas: of the counted form, 0 for a cluster per pair
  int cuts;                       // pairs or CTAs, the fewer
};

// Tiles of 8 query rows where there are more than 4.  A cluster per pair, as large as the places on the GPU allow,
// where that leaves a warp at most 8 units of the longest sequence that the table can hold, or where there are too
// many sequences to count; else counted runs, one CTA a place.
Plan plan(const ifq_kv4_cache& c, int shared) {
  Plan r;
  const int64_t rows = (int64_t)c.n_new * shared;
  r.nt = rows > 4 ? 2 : 1;
  r.qtiles = (int)((rows + 4 * r.nt - 1) / (4 * r.nt));
  const int64_t pairs = (int64_t)c.B * c.kv_heads * r.qtiles, places = 148 * ctas_per_sm(c.dim, r.nt);
  const int64_t units = (c.table_cols * c.page_tokens + kUnit - 1) / kUnit;
  r.cluster = 1;
  while (r.cluster < kMaxCluster && pairs * r.cluster * 2 <= places && r.cluster * kWarps < units) r.cluster *= 2;
  r.ctas = c.B <= kMaxSeqs && (units > r.cluster * kWarps * 8 || pairs > places) ? (int)places : 0;
  if (r.ctas) r.cluster = 1;
  r.cuts = (int)(pairs < r.ctas ? pairs : r.ctas);
  return r;
}

// Partial results of the counted form, rows.
int64_t partials(const Plan& r) { return (int64_t)r.ctas * 2 * 4 * r.nt; }

template <int DIM, int NT>
cudaError_t launch_nt(const AttnParams& p, cudaStream_t s) {
  static uint64_t done = 0;
  auto kernel = kv4_attn_kernel<DIM, NT>;
  constexpr int bytes = Layout<DIM, NT>::kBytes;
  cudaError_t e = allow_smem(kernel, bytes, &done);
  if (e != cudaSuccess) return e;
  const dim3 grid = p.counted ? dim3((unsigned)p.counted)
                              : dim3((unsigned)p.cluster, (unsigned)(p.c.kv_heads * p.qtiles), (unsigned)p.c.B);
  return launch_following<AttnParams>(kernel, grid, kThreads, bytes, p.cluster, p, s);
}

template <int DIM>
cudaError_t launch(const AttnParams& p, const Plan& r, cudaStream_t s) {
  cudaError_t e = r.nt == 1 ? launch_nt<DIM, 1>(p, s) : launch_nt<DIM, 2>(p, s);
  if (e != cudaSuccess || !r.ctas) return e;
  // few pairs have many parts each: 8 pairs 40.0 us with 8 warps a row, 41.3 with 4; 128 pairs 41.6 against 40.1
  const dim3 grid((unsigned)r.cuts, 4u * r.nt);
  if (r.cuts <= 32) return launch_following<AttnParams>(kv4_join_kernel<DIM, 8>, grid, 256, 0, 1, p, s);
  return launch_following<AttnParams>(kv4_join_kernel<DIM, 4>, grid, 128, 0, 1, p, s);
}

}  // namespace

size_t kv4_attention_workspace_bytes(const ifq_kv4_cache& c, int shared) {
  const Plan r = plan(c, shared);
  return (size_t)partials(r) * (2 * c.dim + 2) * 4 + (size_t)r.ctas * sizeof(Cut);
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
  p.scale2 = fabsf(scale) <= 0x1p127f ? scale * kLog2e : NAN;
  p.shared = shared;
  p.cluster = r.cluster;
  p.counted = r.ctas;
  p.by_pair = r.cuts < r.ctas;
  p.qtiles = r.qtiles;
  p.ws_cut = static_cast<Cut*>(ws);
  p.ws_o = reinterpret_cast<float*>(p.ws_cut + r.ctas);
  p.ws_ml = reinterpret_cast<float2*>(p.ws_o + partials(r) * 2 * c.dim);
  p.status = dev_status;
  if (c.dim == 32) return launch<32>(p, r, s);
  if (c.dim == 64) return launch<64>(p, r, s);
  return launch<128>(p, r, s);
}

}  // namespace ifq

// Decode product of layers with 4-bit weights and group scales, y = R_hat [x_re; x_im] for 1 to 16
// tokens: y[n][r] = sum_groups s[r][group] sum_{k in group} q[r][k] x[n][k].
//
// Each 32-bit word of eight codes becomes four bf16 operand registers holding q 2^-6 exactly
// (q4_common.cuh), x is the B operand as it is, so all products are exact and a group accumulates
// in float32; the group's scale multiplies that sum in float32.
//
// HBM-bound by the codes.  A CTA of 4 warps takes row tiles x a slice of the columns, in stages of 128 columns.  A warp
// takes 64 rows of a stage, so that a tile's x is read from shared memory once for four strips, and runs its own ring of
// asynchronous copies of codes and scales.
//   up to 4 tokens  64 rows a CTA: the warps take the slice's stages in turn, each with a ring of x of its own; no barrier
//                   but the warp's
//   5 to 16         128 rows a CTA: two warps with different rows take the same stages and share a ring of x, which each
//                   fills half of.  They meet at a named barrier (one per pair) every stage, when their copies are in:
//                   behind it both read the stage, and neither has still to read the one that is filled next
// The warps' sums are added in shared memory at the end, and where a layer has few row tiles its
// columns are split over a cluster, whose CTAs add theirs through distributed shared memory: one launch,
// no workspace, a fixed order of sums.
//
// Bound: a word takes 5 integer, 4 bf16 and 1 (2 above 8 tokens) matrix instructions and with loads, scales and
// copies 16 to 20 issue slots.  Times are of calls captured in one graph, over weights that L2 does not hold.  One token: a
// 7B-shaped block (105 MB) 20.7 us, 78 % of the copy rate, a 70B-shaped layer set (442 MB) 78 us, 88 %; the rest is start
// and end.  50021 x 4096 in groups of 32, 5 tokens: 25.4 us, 71 % (a group costs 7 instructions per 2 words).  16 tokens:
// the block 41 us, the layer set 116 us, 60 %, by latency: a word's expansion, products and scaling follow one another,
// and the registers leave 12 to 16 warps an SM to cover that (issue 47 %, tensor pipe 36 %, the first stall a fixed wait).
// The registers spilled up to 4 tokens are read 21 times a warp in the block, 0.5 % of its instructions.
#include "ifq_internal.h"
#include "q4_common.cuh"

namespace ifq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStrips = 4;                 // 16-row strips of a warp
constexpr int kCols = 128;                 // of a stage: two tiles
constexpr int kSplits = 4;                 // a layer's columns are split over 1, 2, 4 or 8 CTAs

struct LArg {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* x[2];
  float* y[2];
  int64_t rows;
  int64_t x_split, y_split;  // first column / row of the second plane (cols / rows where there is none)
  int32_t cols;
  int32_t cluster_begin;     // first cluster of the layer in the call
  int32_t split;             // CTAs that share a row tile's columns: 1 .. cluster size, a power of two
  int32_t tiles;             // row tiles
};

template <int kCap>
struct LParams {
  LArg l[kCap];
  int count, B, cluster;
  uint32_t* status;
};

// A stage: two 64-column tiles of a warp's strips, their scales and the x of up to XB tokens.  Above 4 tokens the x of
// a stage is half a warp's codes or more, so two warps with different rows take the same columns and share it (half
// the copies of x: 72 us against 74.6 us for the 70B-shaped gate and down layers at 16 tokens, 54.5 us against 59.1 us
// at 8).  Up to 4 tokens every warp has its own.
template <int G, int XB>
struct Ring {
  static constexpr int NT = (XB + 7) / 8;
  static constexpr int kRowWarps = XB > 4 ? 2 : 1;                      // warps with the same columns
  static constexpr int kColWarps = kWarps / kRowWarps;
  static constexpr int kRows = kRowWarps * kStrips * 16;                // of a CTA
  static constexpr int kStripBytes = 2 * kQ4TileBytes;
  static constexpr int kScaleBytes = kCols / G * 32;                    // of a strip
  static constexpr int kCodes = kStrips * kStripBytes;
  static constexpr int kScales = kStrips * kScaleBytes;
  static constexpr int kX = XB * kCols * 2;
  static constexpr int kStage = kCodes + kScales;
  static constexpr int kStages = 2;
  static constexpr int kXRing = kWarps * kStages * kStage;              // offset of the x rings
  static constexpr int kBytes = kXRing + kColWarps * kStages * kX;
  // CTAs that an SM holds, which the registers are cut to.  Above 8 tokens: 4 (128 registers: 117 us for a 70B-shaped
  // layer set at 16 tokens, 135 us with 3), but 3 for groups of 32, whose scales take more (162 registers: 50021 x 4096
  // at 16 tokens 37 us, 40 us with 4).  5 to 8: 4 (a 7B-shaped block 29.6 us at 8 tokens, 32.0 us with 5 for groups of
  // 64 and more).  Up to 4: 5.
  static constexpr int kCtas = XB > 8 ? (G == 32 ? 3 : 4) : XB > 4 ? 4 : 5;
  static_assert(kCtas * (kBytes + 1024) <= 227 * 1024, "shared memory of an SM");
  static_assert(kBytes >= kColWarps * kRows * XB * 4, "the sums reuse the ring");
};

IFQ_DEVINL uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
IFQ_DEVINL float ld_cluster(const void* smem, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <int G, int XB, int kCap>
__global__ void __launch_bounds__(kThreads, (Ring<G, XB>::kCtas))
    w4_gemv_kernel(const __grid_constant__ LParams<kCap> p) {
  using R = Ring<G, XB>;
  constexpr int NT = R::NT, kRows = R::kRows, kColWarps = R::kColWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
  const int cl = (int)blockIdx.x / p.cluster;
  int li = 0;
  while (li + 1 < p.count && cl >= p.l[li + 1].cluster_begin) ++li;
  const LArg& L = p.l[li];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // this CTA's rows, and its columns [kb, ke) in whole stages; this warp's stages are col_warp, + kColWarps, ...
  const int sub = rank % L.split;
  const int tile = (cl - L.cluster_begin) * (p.cluster / L.split) + rank / L.split;
  const int64_t row0 = (int64_t)tile * kRows;
  const int units = (L.cols + kCols - 1) / kCols, per = (units + L.split - 1) / L.split;
  const int kb = min(units, sub * per) * kCols, ke = tile < L.tiles ? min(L.cols, kb + per * kCols) : kb;
  const int row_warp = warp % R::kRowWarps, col_warp = warp / R::kRowWarps;
  const int k_first = kb + col_warp * kCols;

  // Sources of this lane's copies, moved on to the warp's next stage after each.  Strips past the layer repeat its
  // last one.
  const int64_t strips = (L.rows + 15) / 16, strip0 = row0 / 16 + row_warp * kStrips;
  const uint8_t* code_src[kStrips];
#pragma unroll
  for (int m = 0; m < kStrips; ++m)
    code_src[m] = L.codes + min(strips - 1, strip0 + m) * (L.cols * 8ll) + k_first * 8ll + lane * 16;
  constexpr int kLanes = R::kScaleBytes / 16;                 // lanes that fetch a strip's scales
  const uint8_t* scale_src = reinterpret_cast<const uint8_t*>(L.scales) +
                             min(strips - 1, strip0 + lane / kLanes) * (L.cols / G * 32ll) + k_first / G * 32 +
                             (lane % kLanes) * 16;
  constexpr int kXTokens = 2 * R::kRowWarps;                  // tokens that the warps of a column fetch at a time
  const int xt = (lane >> 4) + 2 * row_warp, xv = lane & 15;  // 8 columns of the tokens xt + kXTokens i
  int xk = k_first + xv * 8;
  bool second = xk >= L.x_split;
  const uint16_t* x_src = second ? L.x[1] + xt * (L.cols - L.x_split) + (xk - L.x_split) : L.x[0] + xt * L.x_split + xk;
  int64_t x_step = kXTokens * (second ? L.cols - L.x_split : L.x_split);
  const uint32_t ring = smem_u32(smem) + warp * R::kStages * R::kStage;
  follow();
  const uint32_t code_dst = ring + lane * 16, scale_dst = ring + R::kCodes + lane * 16;
  const uint32_t x_dst = smem_u32(smem) + R::kXRing + col_warp * R::kStages * R::kX +
                         ((xv >> 2) * XB * 4 + (xv & 3)) * 16 + xt * 64;
  int kl = k_first;   // columns of the next load
  auto load = [&](int slot) {
    if (kl < ke) {
      const bool whole = kl + kCols <= ke;  // a layer's last stage may be one tile
#pragma unroll
      for (int m = 0; m < kStrips; ++m) {
        const uint32_t dst = code_dst + slot * R::kStage + m * R::kStripBytes;
        cp_async16(dst, code_src[m]);
        if (whole) cp_async16(dst + kQ4TileBytes, code_src[m] + kQ4TileBytes);
        code_src[m] += kColWarps * R::kStripBytes;
      }
      if (lane < kStrips * kLanes && (whole || (lane % kLanes) * 16 < 64 / G * 32))
        cp_async16(scale_dst + slot * R::kStage, scale_src);
      scale_src += kColWarps * R::kScaleBytes;
      if (xk < ke) {
        const uint16_t* src = x_src;
#pragma unroll
        for (int i = 0; i < (XB + kXTokens - 1) / kXTokens; ++i) {
          if (kXTokens * i >= p.B) break;
          if (xt + kXTokens * i < p.B) cp_async16(x_dst + slot * R::kX + i * kXTokens * 64, src);
          src += x_step;
        }
      }
      kl += kColWarps * kCols;
      xk += kColWarps * kCols;
      x_src += kColWarps * kCols;
      if (!second && xk >= L.x_split) {
        second = true;
        x_src = L.x[1] + xt * (L.cols - L.x_split) + (xk - L.x_split);
        x_step = kXTokens * (L.cols - L.x_split);
      }
    }
    cp_async_commit();
  };

  float acc[kStrips][NT][4];
#pragma unroll
  for (int m = 0; m < kStrips; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.0f;
  // Columns of B past the last token repeat it (their results are dropped), so that no lane waits on a branch.
  const uint8_t* base0 = smem + warp * R::kStages * R::kStage;
  const uint8_t* xs[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xs[nt] = smem + R::kXRing + col_warp * R::kStages * R::kX + (min(nt * 8 + g, p.B - 1) * 4 + t) * 16;

  auto tile_product = [&](int slot, int i) {
    uint4 b[2][NT];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        b[c][nt] = *reinterpret_cast<const uint4*>(xs[nt] + slot * R::kX + (2 * i + c) * XB * 64);
#pragma unroll
    for (int m = 0; m < kStrips; ++m) {
      const uint4 w4 = *reinterpret_cast<const uint4*>(base0 + lane * 16 + slot * R::kStage + m * R::kStripBytes +
                                                       i * kQ4TileBytes);
      float part[NT][4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t lo[4], hi[4];
        q4_expand(c ? w4.z : w4.x, lo);
        q4_expand(c ? w4.w : w4.y, hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (c == 0 || G == 32) mma_bf16_first(part[nt], lo[0], hi[0], lo[1], hi[1], b[c][nt].x, b[c][nt].y);
          else mma_bf16(part[nt], lo[0], hi[0], lo[1], hi[1], b[c][nt].x, b[c][nt].y);
          mma_bf16(part[nt], lo[2], hi[2], lo[3], hi[3], b[c][nt].z, b[c][nt].w);
        }
        if (c == 1 || G == 32) {
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(base0 + g * 4 + slot * R::kStage + R::kCodes +
                                                                 m * R::kScaleBytes + (64 * i + 32 * c) / G * 32);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[m][nt][0] = fmaf(bf16_lo(sc), part[nt][0], acc[m][nt][0]);
            acc[m][nt][1] = fmaf(bf16_lo(sc), part[nt][1], acc[m][nt][1]);
            acc[m][nt][2] = fmaf(bf16_hi(sc), part[nt][2], acc[m][nt][2]);
            acc[m][nt][3] = fmaf(bf16_hi(sc), part[nt][3], acc[m][nt][3]);
          }
        }
      }
    }
  };

#pragma unroll
  for (int st = 0; st < R::kStages - 1; ++st) load(st);
  for (int k = k_first; k < ke;) {
#pragma unroll
    for (int slot = 0; slot < R::kStages; ++slot, k += kColWarps * kCols) {
      if (k >= ke) break;
      cp_async_wait<R::kStages - 2>();
      // every lane's copies of the stage are in, and the previous stage has been read
      if constexpr (R::kRowWarps == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + col_warp), "n"(32 * R::kRowWarps) : "memory");
      load((slot + R::kStages - 1) % R::kStages);
      tile_product(slot, 0);
      if (k + kCols <= ke) tile_product(slot, 1);
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // sums[col_warp][n][row] in the ring's memory; added over the columns' warps, then over the cluster
  float* sums = reinterpret_cast<float*>(smem);
  const int plane = p.B * kRows;
#pragma unroll
  for (int m = 0; m < kStrips; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = nt * 8 + 2 * t + (e & 1);
        const int row = (row_warp * kStrips + m) * 16 + g + 8 * (e >> 1);
        if (n < p.B) sums[col_warp * plane + n * kRows + row] = acc[m][nt][e];
      }
  __syncthreads();
  auto column_sum = [&](const float* at) {
    if constexpr (kColWarps == 2) return at[0] + at[plane];
    else return (at[0] + at[plane]) + (at[2 * plane] + at[3 * plane]);
  };
  if (p.cluster > 1) {
    for (int i = threadIdx.x; i < plane; i += kThreads) sums[i] = column_sum(sums + i);
    cluster_sync();
  }
  bool bad = false;
  const int span = kRows / L.split;
  for (int i = threadIdx.x; i < p.B * span; i += kThreads) {
    const int n = i / span, lr = sub * span + i % span;
    const int64_t r = row0 + lr;
    if (r >= L.rows) continue;
    float v;
    const float* at = sums + n * kRows + lr;
    if (L.split > 1) {
      v = 0.0f;
      for (int k = 0; k < L.split; ++k) v += ld_cluster(at, rank - sub + k);
    } else {
      v = p.cluster > 1 ? at[0] : column_sum(at);
    }
    v *= kQ4Unit;
    bad |= !(fabsf(v) <= 3.402823466e38f);
    if (r < L.y_split) L.y[0][n * L.y_split + r] = v;
    else L.y[1][n * (L.rows - L.y_split) + r - L.y_split] = v;
  }
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while its sums are being read
}

// When the CTAs of a launch end: the places on the GPU by the time at which each is free.
struct Ends {
  static constexpr int kMax = 24;
  int64_t at[kMax], places[kMax];
  int n = 1;
  explicit Ends(int64_t all) : at{0}, places{all} {}
  // `count` CTAs that take `time` each go to the places that are free first.
  void run(int64_t count, int64_t time) {
    while (count > 0) {
      int first = 0;
      int64_t all = 0;
      for (int i = 0; i < n; ++i) {
        if (at[i] < at[first]) first = i;
        all += places[i];
      }
      if (count >= 4 * all || n == kMax) {  // whole rounds of many CTAs
        const int64_t rounds = count / all > 1 ? count / all : 1;
        for (int i = 0; i < n; ++i) at[i] += rounds * time;
        count -= rounds * all;
        continue;
      }
      const int64_t m = count < places[first] ? count : places[first];
      if (m == places[first]) {
        at[first] += time;
      } else {
        places[first] -= m;
        at[n] = at[first] + time;
        places[n++] = m;
      }
      count -= m;
    }
  }
  int64_t last() const {
    int64_t t = 0;
    for (int i = 0; i < n; ++i) t = at[i] > t ? at[i] : t;
    return t;
  }
};

template <int G, int XB, int kCap>
cudaError_t launch(const ifq_w4_layer* Ls, int count, int B, uint32_t* dev_status, cudaStream_t s) {
  using R = Ring<G, XB>;
  static uint64_t done = 0;
  auto kernel = w4_gemv_kernel<G, XB, kCap>;
  cudaError_t err = allow_smem(kernel, R::kBytes, &done);
  if (err != cudaSuccess) return err;
  // Stages of a warp of layer i where its columns are split over 2^k CTAs, and its row tiles.
  int64_t stages[kCap][kSplits], tiles[kCap], longest = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t units = (Ls[i].cols + kCols - 1) / kCols;
    for (int k = 0; k < kSplits; ++k) stages[i][k] = (units + (R::kColWarps << k) - 1) / (R::kColWarps << k);
    tiles[i] = (Ls[i].rows + R::kRows - 1) / R::kRows;
    longest = stages[i][0] > longest ? stages[i][0] : longest;
  }
  // (All of it on the host, in every call: 0.2 us for one layer, 0.9 for a block of 7, 43 for 32 layers of 32 widths.)
  // How far to split the columns: to slices of at most `len` stages.  Splitting further helps while CTAs are few or
  // long ones end last, and costs every CTA its start and join (kStart stages' time): of the lengths that some layer
  // can be cut to, the one whose CTAs, started longest first on the GPU's places, end first.
  constexpr int kStart = 6;
  auto split_for = [&](int i, int64_t len) {
    int k = 0;
    while (k + 1 < kSplits && stages[i][k] > len) ++k;
    return k;
  };
  int64_t best = longest, best_end = 0;
  for (int c = 0; c < count * kSplits; ++c) {
    const int64_t len = stages[c / kSplits][c % kSplits];
    bool seen = false;
    for (int e = 0; e < c && !seen; ++e) seen = stages[e / kSplits][e % kSplits] == len;
    if (seen) continue;
    Ends ends(148 * R::kCtas);
    for (int64_t top = longest + 1;;) {  // the CTAs of each length, longest first
      int64_t next = 0, n = 0;
      for (int i = 0; i < count; ++i) {
        const int k = split_for(i, len);
        const int64_t st = stages[i][k];
        if (st < top && st > next) next = st, n = 0;
        if (st == next) n += tiles[i] << k;
      }
      if (next == 0) break;
      ends.run(n, next + kStart);
      top = next;
    }
    if (best_end == 0 || ends.last() < best_end) {
      best = len;
      best_end = ends.last();
    }
  }
  int split[kCap], cluster = 1;
  for (int i = 0; i < count; ++i) {
    split[i] = split_for(i, best);
    cluster = (1 << split[i]) > cluster ? 1 << split[i] : cluster;
  }
  // the longest slices first, so that the last CTAs to start are short ones
  int order[kCap];
  for (int i = 0; i < count; ++i) {
    int j = i;
    for (; j > 0 && stages[order[j - 1]][split[order[j - 1]]] < stages[i][split[i]]; --j) order[j] = order[j - 1];
    order[j] = i;
  }
  LParams<kCap> p;
  p.count = count;
  p.B = B;
  p.cluster = cluster;
  p.status = dev_status;
  int64_t clusters = 0;
  for (int i = 0; i < count; ++i) {
    const ifq_w4_layer& a = Ls[order[i]];
    LArg& l = p.l[i];
    l.codes = a.codes;
    l.scales = a.scales;
    l.x[0] = a.x_re;
    l.x[1] = a.x_im;
    l.y[0] = a.y_re;
    l.y[1] = a.y_im;
    l.rows = a.rows;
    l.cols = (int32_t)a.cols;
    l.x_split = a.x_im ? a.cols / 2 : a.cols;
    l.y_split = a.y_im ? a.rows / 2 : a.rows;
    l.split = 1 << split[order[i]];
    l.tiles = (int32_t)tiles[order[i]];
    l.cluster_begin = (int32_t)clusters;
    const int64_t each = cluster / l.split;  // row tiles of a cluster
    clusters += (l.tiles + each - 1) / each;
  }
  return launch_following<LParams<kCap>>(kernel, dim3((unsigned)(clusters * cluster)), kThreads, R::kBytes, cluster, p, s);
}

template <int G, int kCap>
cudaError_t by_batch(const ifq_w4_layer* Ls, int count, int B, uint32_t* dev_status, cudaStream_t s) {
  if (B <= 2) return launch<G, 2, kCap>(Ls, count, B, dev_status, s);
  if (B <= 4) return launch<G, 4, kCap>(Ls, count, B, dev_status, s);
  if (B <= 8) return launch<G, 8, kCap>(Ls, count, B, dev_status, s);
  return launch<G, 16, kCap>(Ls, count, B, dev_status, s);
}

template <int G>
cudaError_t by_count(const ifq_w4_layer* Ls, int count, int B, uint32_t* dev_status, cudaStream_t s) {
  if (count <= 8) return by_batch<G, 8>(Ls, count, B, dev_status, s);
  return by_batch<G, IFQ_MAX_GROUP>(Ls, count, B, dev_status, s);
}

}  // namespace

cudaError_t launch_w4_gemv(const ifq_w4_layer* Ls, int count, int group, int B, uint32_t* dev_status, cudaStream_t s) {
  if (group == 32) return by_count<32>(Ls, count, B, dev_status, s);
  if (group == 64) return by_count<64>(Ls, count, B, dev_status, s);
  return by_count<128>(Ls, count, B, dev_status, s);
}

}  // namespace ifq

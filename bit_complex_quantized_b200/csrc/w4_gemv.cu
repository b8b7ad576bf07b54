// Decode product of layers with 4-bit weights and group scales, y = R_hat [x_re; x_im] for 1 to 16
// tokens: y[n][r] = sum_groups s[r][group] sum_{k in group} q[r][k] x[n][k].
//
// Each 32-bit word of eight codes becomes four bf16 operand registers holding q 2^-6 exactly
// (q4_common.cuh), x is the B operand as it is, so all products are exact and a group accumulates
// in float32; the group's scale multiplies that sum in float32.
//
// HBM-bound by the codes.  A CTA of 8 warps takes 128 kMT rows (16 kMT per warp) x a slice of the
// columns, 256 columns a stage, through a ring of asynchronous copies: codes and scales are contiguous
// runs private to a warp, the stage's x is shared by the CTA (one barrier a stage).  A layer with few row
// tiles has its columns split over a cluster, whose CTAs add their sums through distributed
// shared memory in rank order: one launch, no workspace, a fixed order of sums.
#include "ifq_internal.h"
#include "q4_common.cuh"

namespace ifq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStageCols = 256;
constexpr int kMaxCluster = 8;

struct LArg {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* x[2];
  float* y[2];
  int64_t rows, cols;
  int64_t x_split, y_split;  // first column / row of the second plane (cols / rows where there is none)
  int64_t tile_begin;        // first row tile of the layer in the call
};

template <int kCap>
struct LParams {
  LArg l[kCap];
  int count, B, cluster;
  uint32_t* status;
};

template <int G, int NT, int MT>
struct Ring {
  static constexpr int kScaleBytes = kStageCols / G * 32;               // of a strip of 16 rows
  static constexpr int kStripBytes = kStageCols / 64 * kQ4TileBytes;    // codes of a strip
  static constexpr int kCodes = kWarps * MT * kStripBytes;
  static constexpr int kScales = kWarps * MT * kScaleBytes;
  static constexpr int kX = kStageCols / 32 * NT * 8 * 64;
  static constexpr int kStage = kCodes + kScales + kX;
  static constexpr int kStages = 4;
  static constexpr int kBytes = kStages * kStage;
  static_assert(kBytes >= kWarps * MT * 16 * NT * 8 * 4, "the sums reuse the ring");
};

IFQ_DEVINL uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
IFQ_DEVINL void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
IFQ_DEVINL float ld_cluster(const void* smem, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <int G, int NT, int MT, int kCap>
__global__ void __launch_bounds__(kThreads) w4_gemv_kernel(const __grid_constant__ LParams<kCap> p) {
  using R = Ring<G, NT, MT>;
  constexpr int U = G > 64 ? G : 64;
  constexpr int kRows = kWarps * MT * 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
  const int64_t tile = (int64_t)blockIdx.x / p.cluster;
  int li = 0;
  while (li + 1 < p.count && tile >= p.l[li + 1].tile_begin) ++li;
  const LArg& L = p.l[li];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = (tile - L.tile_begin) * kRows;
  const int64_t strips = (L.rows + 15) / 16, strip0 = row0 / 16 + warp * MT;
  // this CTA's columns, whole units
  const int64_t units = L.cols / U, per = (units + p.cluster - 1) / p.cluster;
  const int64_t kb = min(units, rank * per) * U, ke = min(units, (rank + 1) * per) * U;

  // Sources of this thread's copies, moved on by a stage after each: its strips' codes and scales, and 8
  // columns of the tokens warp + 8 i (in the first plane up to x_split, then in the second).
  const uint8_t* code_src[MT];
  const uint8_t* scale_src[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t strip = min(strip0 + m, strips - 1);   // rows past the layer repeat its last strip
    code_src[m] = L.codes + (strip * (L.cols / 64) + kb / 64) * kQ4TileBytes + lane * 16;
    scale_src[m] = reinterpret_cast<const uint8_t*>(L.scales) + (strip * (L.cols / G) + kb / G) * 32 + lane * 16;
  }
  int64_t xk = kb + lane * 8;
  int64_t k_left = ke - kb;   // columns not yet asked for
  int slot = 0;               // of the next load
  auto load = [&]() {
    if (k_left > 0) {
      uint8_t* base = smem + slot * R::kStage;
      const int tiles = k_left >= kStageCols ? kStageCols / 64 : (int)(k_left / 64);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint8_t* c = base + (warp * MT + m) * R::kStripBytes + lane * 16;
#pragma unroll
        for (int i = 0; i < kStageCols / 64; ++i)
          if (i < tiles) cp_async16(c + i * kQ4TileBytes, code_src[m] + i * kQ4TileBytes);
        if (lane * 16 < tiles * 64 / G * 32)
          cp_async16(base + R::kCodes + (warp * MT + m) * R::kScaleBytes + lane * 16, scale_src[m]);
        code_src[m] += R::kStripBytes;
        scale_src[m] += R::kScaleBytes;
      }
      uint8_t* xs = base + R::kCodes + R::kScales + ((lane >> 2) * NT * 32 + (lane & 3)) * 16;
      const bool second = xk >= L.x_split;
      const uint16_t* src = second ? L.x[1] + (xk - L.x_split) : L.x[0] + xk;
      const int64_t width = second ? L.cols - L.x_split : L.x_split;
      if (xk < ke)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (warp + 8 * i < p.B) cp_async16(xs + (warp + 8 * i) * 64, src + (warp + 8 * i) * width);
      xk += kStageCols;
      k_left -= kStageCols;
      slot = slot + 1 == R::kStages ? 0 : slot + 1;
    }
    cp_async_commit();
  };

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.0f;

  // Columns of B past the last token repeat it (their results are dropped), so that no lane waits on a branch.
  int x_off[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x_off[nt] = (min(nt * 8 + g, p.B - 1) * 4 + t) * 16;

  auto unit = [&](const uint8_t* base, int u) {
    const uint8_t* cs = base + warp * MT * R::kStripBytes + lane * 16;
    const uint8_t* ss = base + R::kCodes + warp * MT * R::kScaleBytes + g * 4;
    const uint8_t* xs = base + R::kCodes + R::kScales;
    float part[MT][NT][4];
#pragma unroll
    for (int i = 0; i < U / 64; ++i) {
      const int tl = u * (U / 64) + i;
      uint4 w4[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        w4[m] = *reinterpret_cast<const uint4*>(cs + m * R::kStripBytes + tl * kQ4TileBytes);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int ch = tl * 2 + c;
        uint4 b[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt] = *reinterpret_cast<const uint4*>(xs + ch * NT * 512 + x_off[nt]);
        const bool first = (64 * i + 32 * c) % G == 0, last = (64 * i + 32 * c + 32) % G == 0;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t lo[4], hi[4];
          q4_expand<kQ4Sub8>(c ? w4[m].z : w4[m].x, lo);
          q4_expand<kQ4Sub8>(c ? w4[m].w : w4[m].y, hi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (first) mma_bf16_first(part[m][nt], lo[0], hi[0], lo[1], hi[1], b[nt].x, b[nt].y);
            else mma_bf16(part[m][nt], lo[0], hi[0], lo[1], hi[1], b[nt].x, b[nt].y);
            mma_bf16(part[m][nt], lo[2], hi[2], lo[3], hi[3], b[nt].z, b[nt].w);
          }
          if (last) {
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(ss + m * R::kScaleBytes + (ch * 32 / G) * 32);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              acc[m][nt][0] = fmaf(bf16_lo(sc), part[m][nt][0], acc[m][nt][0]);
              acc[m][nt][1] = fmaf(bf16_lo(sc), part[m][nt][1], acc[m][nt][1]);
              acc[m][nt][2] = fmaf(bf16_hi(sc), part[m][nt][2], acc[m][nt][2]);
              acc[m][nt][3] = fmaf(bf16_hi(sc), part[m][nt][3], acc[m][nt][3]);
            }
          }
        }
      }
    }
  };

#pragma unroll
  for (int st = 0; st < R::kStages - 1; ++st) load();
  int at = 0;  // slot of the stage being read
  for (int64_t left = ke - kb; left > 0; left -= kStageCols) {
    cp_async_wait<R::kStages - 2>();
    __syncthreads();  // the stage's copies of every warp are in; the previous stage has been read
    load();
    const uint8_t* base = smem + at * R::kStage;
    at = at + 1 == R::kStages ? 0 : at + 1;
    if (left >= kStageCols) {
#pragma unroll
      for (int u = 0; u < kStageCols / U; ++u) unit(base, u);
    } else {
      for (int u = 0; u < (int)(left / U); ++u) unit(base, u);
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // sums[n][row] in the ring's memory, then over the cluster
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = nt * 8 + 2 * t + (e & 1);
        if (n < p.B) sums[n * kRows + (warp * MT + m) * 16 + g + 8 * (e >> 1)] = acc[m][nt][e];
      }
  if (p.cluster > 1) cluster_sync();
  else __syncthreads();
  bool bad = false;
  const int span = kRows / p.cluster;
  for (int i = threadIdx.x; i < p.B * span; i += kThreads) {
    const int n = i / span, lr = rank * span + i % span;
    const int64_t r = row0 + lr;
    if (r >= L.rows) continue;
    float v = 0.0f;
    if (p.cluster > 1) {
      for (int k = 0; k < p.cluster; ++k) v += ld_cluster(sums + n * kRows + lr, k);
    } else {
      v = sums[n * kRows + lr];
    }
    v *= kQ4Unit;
    bad |= !(fabsf(v) <= 3.402823466e38f);
    if (r < L.y_split) L.y[0][n * L.y_split + r] = v;
    else L.y[1][n * (L.rows - L.y_split) + r - L.y_split] = v;
  }
  if (bad) set_status(p.status, IFQ_DEV_NONFINITE);
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while its sums are being read
}

// The kernel's shared memory above 48 KB has to be allowed once per device.
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

template <int G, int NT, int MT, int kCap>
cudaError_t launch(const ifq_w4_layer* Ls, int count, int B, uint32_t* dev_status, cudaStream_t s) {
  using R = Ring<G, NT, MT>;
  static uint64_t done = 0;
  auto kernel = w4_gemv_kernel<G, NT, MT, kCap>;
  cudaError_t err = allow_smem(kernel, R::kBytes, &done);
  if (err != cudaSuccess) return err;
  LParams<kCap> p;
  p.count = count;
  p.B = B;
  p.status = dev_status;
  constexpr int kRows = kWarps * MT * 16;
  // the layers with the longest rows first, so that the last CTAs to start are short ones
  int order[kCap];
  for (int i = 0; i < count; ++i) {
    int j = i;
    for (; j > 0 && Ls[order[j - 1]].cols < Ls[i].cols; --j) order[j] = order[j - 1];
    order[j] = i;
  }
  int64_t tiles = 0;
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
    l.cols = a.cols;
    l.x_split = a.x_im ? a.cols / 2 : a.cols;
    l.y_split = a.y_im ? a.rows / 2 : a.rows;
    l.tile_begin = tiles;
    tiles += (a.rows + kRows - 1) / kRows;
  }
  int cluster = 1;
  while (cluster < kMaxCluster && tiles * cluster < 148 * 2) cluster *= 2;
  p.cluster = cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = R::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int G, int kCap>
cudaError_t by_batch(const ifq_w4_layer* Ls, int count, int B, uint32_t* dev_status, cudaStream_t s) {
  if (B <= 8) return launch<G, 1, 1, kCap>(Ls, count, B, dev_status, s);
  return launch<G, 2, 2, kCap>(Ls, count, B, dev_status, s);
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

// Root-mean-square norm in front of the GEMM, and its gradient.
//
// Forward, per row of the residual stream:
//   h    = x + residual, rounded to the stream's type (h = x without residual);
//   rstd = 1 / sqrt(mean(h^2) + eps);
//   y    = h * rstd * weight;
// and per g x g block of y, as the quantiser does it:
//   s = amax |y| / FMAX (1 if that is 0),  q = FP8 code of y / s.
// y exists only in registers: the outputs are h, q, s and rstd.
//
// Backward, from the gradient dy of y (n = h * rstd):
//   dn = dy * weight,  dx = rstd * (dn - n * mean(dn * n)) [+ dresidual],
//   dweight[c] = sum over rows of dy * n.
// dx is the gradient of x and of the residual alike; dresidual is what comes
// down the skip path. The quantiser is passed straight through.
//
// All of it is memory-bound: 2-byte streams of 3 reads or writes per element
// and a byte of codes forward, 4 backward.
#include <cmath>

#include "bsgemm_host.h"
#include "bsgemm_rows.cuh"

namespace bsgn {

using namespace bsgr;

// ------------------------------------------------------------------ forward
//
// A cluster of C CTAs takes one row of scale blocks (g rows, all columns);
// CTA `rank` takes its blocks rank, rank + C, ... A row's mean square needs
// every CTA's share, so each CTA writes the g partial sums it has into every
// CTA of the cluster (distributed shared memory) and one cluster barrier
// separates two passes over the CTA's blocks:
//   pass 1: h = x + residual, stored, and its squares summed per row;
//   pass 2: h is read again (by the thread that wrote it, from L2), scaled,
//           and the block quantised.
// Splitting the rows by columns this way keeps a block's amax inside one CTA,
// and the only exchange is g floats per CTA. Sums are added in rank order, so
// results do not vary between runs.
//
// A pass over a block takes rp rows at a time, g / 8 threads to a row. With
// fewer rows than the 256 threads could take (a decode step), rp is cut to
// them and the threads left over take other blocks at the same time.

constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  void* stream_out;
  uint8_t* q;
  float* scales;
  float* rstd;
  int64_t rows, cols;
  int col_blocks;
  int cluster;
  int row_log;      // log2 of the rows per pass
  int weight_bf16;
  float eps;
};

__device__ __forceinline__ void load_weight(const NormParams& p, int64_t c, float2 (&w)[4]) {
  if (p.weight_bf16) widen<true>(load_run<true>(p.weight, c), w);
  else               widen<false>(load_run<false>(p.weight, c), w);
}

template <int G, bool BF16, int FMT, bool RES>
__global__ void __launch_bounds__(kThreads, 2) norm_quant_kernel(const __grid_constant__ NormParams p) {
  constexpr int L = G / kVec;          // threads to a row of a block
  constexpr int RP = kThreads / L;     // rows the CTA takes at a time (rp at most)
  constexpr int NP = G / RP;           // passes over a full block
  // passes loaded at a time, so that many loads are in flight at once; where
  // they cover the block its values also stay in registers for the encoding
  constexpr int U = NP < (BF16 ? 8 : 4) ? NP : (BF16 ? 8 : 4);
  constexpr bool kHeld = U == NP;
  __shared__ float part[kMaxCluster][G];  // the row sums of each CTA of the cluster
  __shared__ float own_sum[G];
  __shared__ float row_rstd[G];
  __shared__ uint32_t block_max[3][kThreads / L];

  const int tid = threadIdx.x;
  const int rank = p.cluster > 1 ? static_cast<int>(bsg::cluster_ctarank()) : 0;
  const int64_t rb = blockIdx.x / p.cluster;
  const int64_t r0 = rb * G;
  const int rows = static_cast<int>(p.rows - r0 < G ? p.rows - r0 : G);
  const int rp = 1 << p.row_log;
  const int slots = RP >> p.row_log;   // blocks taken at the same time
  const int col8 = (tid % L) * kVec;
  const int rr = (tid / L) & (rp - 1);
  const int slot = (tid / L) >> p.row_log;
  const int step = p.cluster * slots;  // col_blocks + step stays far below 2^31

  if (tid < 3 * RP) (&block_max[0][0])[tid] = 0;
  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();

  // ---- pass 1
  float ss[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) ss[j] = 0.f;
  for (int b = rank + p.cluster * slot; b < p.col_blocks; b += step) {
    const int64_t c = static_cast<int64_t>(b) * G + col8;
    if (c >= p.cols) continue;
#pragma unroll
    for (int j0 = 0; j0 < NP; j0 += U) {
      Run<BF16> xr[U], res[RES ? U : 1];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int r = rr + (j0 + j) * rp;
        xr[j] = zero_run<BF16>();
        if constexpr (RES) res[j] = zero_run<BF16>();
        if (r < rows) {
          xr[j] = load_run<BF16>(p.x, (r0 + r) * p.cols + c);
          if constexpr (RES) res[j] = load_run<BF16>(p.residual, (r0 + r) * p.cols + c);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int r = rr + (j0 + j) * rp;
        float2 v[4];
        widen<BF16>(xr[j], v);
        if constexpr (RES) {
          float2 u[4];
          widen<BF16>(res[j], u);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = add2(v[i], u[i]);
          // the stream is rounded to its type here, once, and it is the
          // rounded stream that is normalised: the next layer and the
          // backward pass read the same values
          const Run<BF16> h = narrow<BF16>(v);
          if (r < rows) store_run<BF16>(p.stream_out, (r0 + r) * p.cols + c, h);
          widen<BF16>(h, v);
        }
        float2 s = mul2(v[0], v[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s = bsg::ffma2(v[i], v[i], s);
        ss[j0 + j] += s.x + s.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NP; ++j) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
    // row rr + j * rp of slot 0..slots-1; where rp < RP only j = 0 has rows
    if (tid % L == 0 && (rp == RP || j == 0)) own_sum[j * RP + tid / L] = ss[j];
  }
  __syncthreads();
  for (int r = tid; r < rows; r += kThreads) {
    float s = own_sum[r];
    for (int k = 1; k < slots; ++k) s += own_sum[k * rp + r];
    if (p.cluster == 1) {
      part[0][r] = s;
    } else {
      const uint32_t mine = bsg::smem_addr(&part[rank][r]);
      for (int d = 0; d < p.cluster; ++d) st_cluster_f32(bsg::mapa_shared(mine, d), s);
    }
  }
  // every thread of the cluster arrives, also in CTAs without blocks; after it
  // no CTA touches another's shared memory, so any may run on to its exit
  __syncwarp();
  if (p.cluster > 1) bsg::cluster_sync_all();
  else __syncthreads();
  for (int r = tid; r < rows; r += kThreads) {
    float s = part[0][r];
    for (int k = 1; k < p.cluster; ++k) s += part[k][r];
    const float v = __frsqrt_rn(s / static_cast<float>(p.cols) + p.eps);
    row_rstd[r] = v;
    if (rank == 0 && p.rstd != nullptr) p.rstd[r0 + r] = v;
  }
  __syncthreads();

  // ---- pass 2
  const void* h_src = RES ? p.stream_out : p.x;
  int buf = 0;
  for (int base = rank; base < p.col_blocks; base += step) {
    const int b = base + p.cluster * slot;
    const int64_t c = static_cast<int64_t>(b) * G + col8;
    const bool in = b < p.col_blocks && c < p.cols;
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = both(0.f);
    if (in) load_weight(p, c, w);
    Run<BF16> h[U];
    auto load = [&](int j0) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int r = rr + (j0 + j) * rp;
        h[j] = zero_run<BF16>();
        if (in && r < rows) h[j] = load_run<BF16>(h_src, (r0 + r) * p.cols + c);
      }
    };
    // y of the loaded row j0 + j
    auto value = [&](int j0, int j, float2 (&v)[4]) {
      const int r = rr + (j0 + j) * rp;
      const float rs = r < rows ? row_rstd[r] : 0.f;
      widen<BF16>(h[j], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(mul2(v[i], both(rs)), w[i]);
    };
    float amax = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < NP; j0 += U) {
      load(j0);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float2 v[4];
        value(j0, j, v);
        amax = max_abs(amax, v);
      }
    }
    // magnitudes are not negative, so their bit patterns order as they do
    if (slots == 1) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
      if ((tid & 31) == 0) atomicMax(&block_max[buf][0], m);
    } else {
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (tid % L == 0) atomicMax(&block_max[buf][slot], __float_as_uint(amax));
    }
    __syncthreads();
    const Scale s = block_scale<FMT>(__uint_as_float(block_max[buf][slot]));
    // the maxima of the block before this one: every thread has read them, and
    // they are used again only after the next barrier
    if (tid < RP) block_max[buf == 0 ? 2 : buf - 1][tid] = 0;
    buf = buf == 2 ? 0 : buf + 1;
    if (b < p.col_blocks && rr == 0 && col8 == 0) p.scales[rb * p.col_blocks + b] = s.s;
#pragma unroll 1
    for (int j0 = 0; j0 < NP; j0 += U) {
      if constexpr (!kHeld) load(j0);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int r = rr + (j0 + j) * rp;
        float2 v[4];
        value(j0, j, v);
        if (in && r < rows) store_codes<FMT>(p.q + (r0 + r) * p.cols + c, v, s);
      }
    }
  }
}

template <int G, bool BF16, int FMT, bool RES>
bsgemm_status launch_norm(NormParams& p, cudaStream_t stream, const bsg_host::DeviceInfo& dev) {
  auto kern = norm_quant_kernel<G, BF16, FMT, RES>;
  static bsg_host::PerDeviceOnce setup;
  if (!setup.done(dev.ordinal)) {
    // clusters of 16 are beyond the portable size
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return BSGEMM_ERR_CUDA;
    setup.mark(dev.ordinal);
  }
  constexpr int RP = kThreads / (G / kVec);
  p.row_log = 0;
  while ((1 << p.row_log) < RP && (int64_t{1} << p.row_log) < p.rows) ++p.row_log;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && 2 * p.cluster <= p.col_blocks) p.cluster *= 2;
  const int64_t row_blocks = (p.rows + G - 1) / G;
  return launch_rows(kern, row_blocks * p.cluster, kThreads, 0, p.cluster, stream, p);
}

template <int G>
bsgemm_status norm_of(int src, int fmt, NormParams& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  p.col_blocks = static_cast<int>((p.cols + G - 1) / G);
  const bool bf16 = src == BSGEMM_SRC_BF16, e5 = fmt == BSGEMM_FP8_E5M2, res = p.residual != nullptr;
#define BSGN_GO(B, F) \
  return res ? launch_norm<G, B, F, true>(p, st, dev) : launch_norm<G, B, F, false>(p, st, dev)
  if (bf16 && !e5) BSGN_GO(true, BSGEMM_FP8_E4M3);
  if (bf16) BSGN_GO(true, BSGEMM_FP8_E5M2);
  if (!e5) BSGN_GO(false, BSGEMM_FP8_E4M3);
  BSGN_GO(false, BSGEMM_FP8_E5M2);
#undef BSGN_GO
}

// ------------------------------------------------------------------ backward
//
// A row's gradient needs one sum over its columns (dy * weight * h), so a row
// is read once into registers: a cluster of C CTAs takes the columns of a row
// in slices of at most 4096, a run to a thread, and the CTA's 512 threads take
// 512 / TC rows at a time where a slice needs only TC of them. Each thread
// keeps the sums of dy * n of its 8 columns over all its rows; at the end they
// are added over the CTA's row groups and written as one row of partial sums,
// and a second kernel adds those rows in order (no atomics: the order never
// changes).

constexpr int kBwdThreads = 512;
constexpr int kBwdRows = 2;          // rows a thread holds at a time
constexpr int kBwdMaxParts = 512;    // rows of partial sums at most
constexpr int64_t kBwdMaxCols = int64_t{kMaxCluster} * kBwdThreads * kVec;

struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* skip;
  void* dx;
  float* part;       // [parts][cols]
  int64_t rows, cols;
  int cluster;
  int slice;         // columns per CTA, a multiple of 8
  int tc_log;        // log2 of the threads to a row
  int parts;
  int weight_bf16;
};

template <bool BF16, bool SKIP>
__global__ void __launch_bounds__(kBwdThreads, BF16 ? 2 : 1)
    norm_backward_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int R = kBwdRows;
  constexpr int kWarps = kBwdThreads / 32;
  __shared__ float warp_sum[2][R][kWarps];
  __shared__ float cta_sum[2][R][kMaxCluster][kBwdThreads / 32];  // per row group (TC >= 32: at most 16)
  __shared__ float2 dw_sum[kBwdThreads * 4];

  const int tid = threadIdx.x, warp = tid / 32;
  const int rank = p.cluster > 1 ? static_cast<int>(bsg::cluster_ctarank()) : 0;
  const int part = blockIdx.x / p.cluster;
  const int tc = 1 << p.tc_log;
  const int groups = kBwdThreads >> p.tc_log;
  const int group = tid >> p.tc_log;
  const int warps_per_group = tc / 32;
  const int local = (tid & (tc - 1)) * kVec;
  const int64_t c = static_cast<int64_t>(rank) * p.slice + local;
  const bool in_cols = local < p.slice && c < p.cols;

  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();

  float2 w[4], dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = dw[i] = both(0.f);
  if (in_cols) {
    if (p.weight_bf16) widen<true>(load_run<true>(p.weight, c), w);
    else               widen<false>(load_run<false>(p.weight, c), w);
  }
  const float inv_cols = 1.0f / static_cast<float>(p.cols);

  int buf = 0;
  // the part's rows: batches of groups * R, dealt out in turn
  const int64_t batch = static_cast<int64_t>(groups) * R;
  for (int64_t base = part * batch; base < p.rows; base += p.parts * batch) {
    Run<BF16> dy[R], h[R], sk[SKIP ? R : 1];
    float rs[R], dot[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t r = base + j * groups + group;
      dy[j] = h[j] = zero_run<BF16>();
      if constexpr (SKIP) sk[j] = zero_run<BF16>();
      rs[j] = 0.f;
      if (in_cols && r < p.rows) {
        dy[j] = load_run<BF16>(p.dy, r * p.cols + c);
        h[j] = load_run<BF16>(p.h, r * p.cols + c);
        if constexpr (SKIP) sk[j] = load_run<BF16>(p.skip, r * p.cols + c);
        rs[j] = __ldg(p.rstd + r);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float2 a[4], b[4];
      widen<BF16>(dy[j], a);
      widen<BF16>(h[j], b);
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 n = mul2(b[i], both(rs[j]));
        dw[i] = bsg::ffma2(a[i], n, dw[i]);
        s = bsg::ffma2(mul2(a[i], w[i]), n, s);
      }
      dot[j] = s.x + s.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if ((tid & 31) == 0) warp_sum[buf][j][warp] = dot[j];
    }
    __syncthreads();
    if (p.cluster > 1) {
      // (slices of a cluster have 4096 columns at most, half of that at
      // least: tc is 256 or 512 and there are few groups)
      if (tid < R * groups) {
        const int j = tid / groups, g = tid % groups;
        float s = 0.f;
        for (int k = 0; k < warps_per_group; ++k) s += warp_sum[buf][j][g * warps_per_group + k];
        const uint32_t mine = bsg::smem_addr(&cta_sum[buf][j][rank][g]);
        for (int d = 0; d < p.cluster; ++d) st_cluster_f32(bsg::mapa_shared(mine, d), s);
      }
      __syncwarp();
      bsg::cluster_sync_all();
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t r = base + j * groups + group;
      float s = 0.f;
      if (p.cluster > 1) {
        for (int k = 0; k < p.cluster; ++k) s += cta_sum[buf][j][k][group];
      } else {
        for (int k = 0; k < warps_per_group; ++k) s += warp_sum[buf][j][group * warps_per_group + k];
      }
      const float m = s * inv_cols;   // mean(dn * n)
      float2 a[4], b[4];
      widen<BF16>(dy[j], a);
      widen<BF16>(h[j], b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 n = mul2(b[i], both(rs[j]));
        const float2 dn = mul2(a[i], w[i]);
        a[i] = mul2(bsg::ffma2(n, both(-m), dn), both(rs[j]));
      }
      if constexpr (SKIP) {
        widen<BF16>(sk[j], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = add2(a[i], b[i]);
      }
      if (in_cols && r < p.rows) store_run<BF16>(p.dx, r * p.cols + c, narrow<BF16>(a));
    }
    // the sums are double-buffered: a thread writes a buffer again two batches
    // on, past a barrier that follows every read of it
    buf ^= 1;
  }

  // the row groups' sums, added in order by the first group's threads
  const int t = tid & (tc - 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) dw_sum[i * kBwdThreads + tid] = dw[i];
  __syncthreads();
  if (group == 0 && in_cols) {
    for (int g = 1; g < groups; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) dw[i] = add2(dw[i], dw_sum[i * kBwdThreads + (g << p.tc_log) + t]);
    store_run<false>(p.part, static_cast<int64_t>(part) * p.cols + c, narrow<false>(dw));
  }
}

// One CTA adds 32 columns: 32 warps take every 32nd row, then one warp adds
// the 32 sums in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int parts, int64_t cols, float* out) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int i = warp; i < parts; i += 32) s += __ldcg(part + static_cast<int64_t>(i) * cols + c);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += sums[k][lane];
    out[c] = s;
  }
}

// Rows of partial sums that a backward call of `rows` rows can have at most.
int64_t bwd_parts_bound(int64_t rows) { return rows < kBwdMaxParts ? rows : kBwdMaxParts; }

}  // namespace bsgn

namespace bsgr {
bsgemm_status launch_column_sum(const float* part, int parts, int64_t cols, float* out, cudaStream_t stream) {
  return launch_rows(bsgn::column_sum_kernel, (cols + 31) / 32, 1024, 0, 1, stream, part, parts, cols, out);
}
}  // namespace bsgr

extern "C" bsgemm_status bsgemm_rms_norm_quantize_fp8(int src_dtype, int weight_dtype, int fp8_format,
                                                      const void* x, const void* residual, const void* weight,
                                                      float eps, int64_t rows, int64_t cols, int gran,
                                                      void* residual_out, void* q, float* scales, float* rstd,
                                                      bsgemm_stream_t stream) {
  if (!x || !weight || !q || !scales || (residual != nullptr) != (residual_out != nullptr))
    return BSGEMM_ERR_INVALID_ARG;
  if (weight_dtype != BSGEMM_SRC_F32 && weight_dtype != BSGEMM_SRC_BF16) return BSGEMM_ERR_INVALID_ARG;
  if (fp8_format != BSGEMM_FP8_E4M3 && fp8_format != BSGEMM_FP8_E5M2) return BSGEMM_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return BSGEMM_ERR_INVALID_ARG;
  if (gran != 64 && gran != 128 && gran != 256) return BSGEMM_ERR_UNSUPPORTED_GRAN;
  bsgemm_status st = bsgr::check_rows(src_dtype, rows, cols);
  if (st != BSGEMM_OK) return st;
  if (!bsgr::aligned(x, 16) || !bsgr::aligned(residual, 16) || !bsgr::aligned(weight, 16) ||
      !bsgr::aligned(residual_out, 16) || !bsgr::aligned(q, 16) || !bsgr::aligned(scales, 4) ||
      !bsgr::aligned(rstd, 4))
    return BSGEMM_ERR_MISALIGNED;
  {
    using bsgr::Span;
    const size_t n = static_cast<size_t>(rows) * static_cast<size_t>(cols);
    const size_t bytes = n * (src_dtype == BSGEMM_SRC_BF16 ? 2 : 4);
    const Span h{residual_out, bytes}, sx{x, bytes}, sr{residual, bytes};
    const Span sw{weight, static_cast<size_t>(cols) * (weight_dtype == BSGEMM_SRC_BF16 ? 2 : 4)};
    const Span sq{q, n}, ss{scales, bsgr::blocks_bytes(rows, cols, gran)};
    const Span sd{rstd, static_cast<size_t>(rows) * sizeof(float)};
    const Span others[] = {sq, ss, sd}, in[] = {sx, sr, sw, h};
    const Span stream_only[] = {h}, stream_in[] = {bsgr::unless_same(h, sx), bsgr::unless_same(h, sr), sw};
    if (bsgr::any_overlap(others, in) || bsgr::any_overlap(stream_only, stream_in)) return BSGEMM_ERR_INVALID_ARG;
  }
  bsg_host::DeviceInfo dev;
  st = bsg_host::device_info(dev);
  if (st != BSGEMM_OK) return st;
  bsgn::NormParams p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.stream_out = residual_out;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.rstd = rstd;
  p.rows = rows;
  p.cols = cols;
  p.weight_bf16 = weight_dtype == BSGEMM_SRC_BF16;
  p.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (gran) {
    case 64:  return bsgn::norm_of<64>(src_dtype, fp8_format, p, s, dev);
    case 128: return bsgn::norm_of<128>(src_dtype, fp8_format, p, s, dev);
    default:  return bsgn::norm_of<256>(src_dtype, fp8_format, p, s, dev);
  }
}

extern "C" size_t bsgemm_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return static_cast<size_t>(bsgn::bwd_parts_bound(rows)) * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" bsgemm_status bsgemm_rms_norm_backward(int src_dtype, int weight_dtype, const void* dy, const void* h,
                                                  const void* weight, const float* rstd, const void* dresidual,
                                                  int64_t rows, int64_t cols, void* dx, float* dweight,
                                                  void* workspace, size_t workspace_bytes, bsgemm_stream_t stream) {
  if (!dy || !h || !weight || !rstd || !dx || !dweight || !workspace) return BSGEMM_ERR_INVALID_ARG;
  if (weight_dtype != BSGEMM_SRC_F32 && weight_dtype != BSGEMM_SRC_BF16) return BSGEMM_ERR_INVALID_ARG;
  bsgemm_status st = bsgr::check_rows(src_dtype, rows, cols);
  if (st != BSGEMM_OK) return st;
  if (cols > bsgn::kBwdMaxCols) return BSGEMM_ERR_INVALID_ARG;
  if (workspace_bytes < bsgemm_rms_norm_backward_workspace(rows, cols)) return BSGEMM_ERR_INVALID_ARG;
  if (!bsgr::aligned(dy, 16) || !bsgr::aligned(h, 16) || !bsgr::aligned(weight, 16) || !bsgr::aligned(rstd, 4) ||
      !bsgr::aligned(dresidual, 16) || !bsgr::aligned(dx, 16) || !bsgr::aligned(dweight, 16) ||
      !bsgr::aligned(workspace, 16))
    return BSGEMM_ERR_MISALIGNED;
  {
    using bsgr::Span;
    const size_t bytes = static_cast<size_t>(rows) * static_cast<size_t>(cols) * (src_dtype == BSGEMM_SRC_BF16 ? 2 : 4);
    const Span sx{dx, bytes}, sy{dy, bytes}, sh{h, bytes}, sk{dresidual, bytes};
    const Span sw{weight, static_cast<size_t>(cols) * (weight_dtype == BSGEMM_SRC_BF16 ? 2 : 4)};
    const Span sr{rstd, static_cast<size_t>(rows) * sizeof(float)};
    const Span dw{dweight, static_cast<size_t>(cols) * sizeof(float)};
    const Span ws{workspace, bsgemm_rms_norm_backward_workspace(rows, cols)};
    const Span others[] = {dw, ws}, in[] = {sy, sh, sw, sr, sk, sx};
    const Span grad[] = {sx}, grad_in[] = {bsgr::unless_same(sx, sy), bsgr::unless_same(sx, sk), sh, sw, sr};
    if (bsgr::any_overlap(others, in) || bsgr::any_overlap(grad, grad_in)) return BSGEMM_ERR_INVALID_ARG;
  }
  bsg_host::DeviceInfo dev;
  st = bsg_host::device_info(dev);
  if (st != BSGEMM_OK) return st;
  const bool bf16 = src_dtype == BSGEMM_SRC_BF16, skip = dresidual != nullptr;
  bsgn::NormBwdParams p{};
  p.dy = dy;
  p.h = h;
  p.weight = weight;
  p.rstd = rstd;
  p.skip = dresidual;
  p.dx = dx;
  p.rows = rows;
  p.cols = cols;
  p.weight_bf16 = weight_dtype == BSGEMM_SRC_BF16;
  p.cluster = 1;
  while (int64_t{p.cluster} * bsgn::kBwdThreads * bsgr::kVec < cols) p.cluster *= 2;
  const int64_t runs = cols / bsgr::kVec;
  p.slice = static_cast<int>((runs + p.cluster - 1) / p.cluster * bsgr::kVec);
  p.tc_log = 5;
  while ((bsgr::kVec << p.tc_log) < p.slice) ++p.tc_log;
  const int64_t batch = int64_t{bsgn::kBwdThreads >> p.tc_log} * bsgn::kBwdRows;
  const int64_t batches = (rows + batch - 1) / batch;
  int64_t parts = int64_t{dev.num_sms} * (bf16 ? 2 : 1) / p.cluster;
  if (parts < 1) parts = 1;
  if (parts > batches) parts = batches;
  if (parts > bsgn::kBwdMaxParts) parts = bsgn::kBwdMaxParts;
  p.parts = static_cast<int>(parts);
  // one row of partial sums is the result itself
  p.part = parts == 1 ? dweight : static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t grid = parts * p.cluster;
  auto go = [&](auto kern) -> bsgemm_status {
    if (p.cluster > 8) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return BSGEMM_ERR_CUDA;
    }
    return bsgr::launch_rows(kern, grid, bsgn::kBwdThreads, 0, p.cluster, s, p);
  };
  if (bf16) st = skip ? go(bsgn::norm_backward_kernel<true, true>) : go(bsgn::norm_backward_kernel<true, false>);
  else      st = skip ? go(bsgn::norm_backward_kernel<false, true>) : go(bsgn::norm_backward_kernel<false, false>);
  if (st != BSGEMM_OK || parts == 1) return st;
  return bsgr::launch_column_sum(p.part, p.parts, cols, dweight, s);
}

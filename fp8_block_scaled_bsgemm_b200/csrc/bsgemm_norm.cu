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

#include "bsgemm_blocks.cuh"

namespace bsgn {

using namespace bsgr;

// ------------------------------------------------------------------ forward
//
// A row's mean square needs all its columns, a block's amax g rows: the two
// cuts cross, so the work is done in two steps.
//
// Many rows: two kernels. The first streams the rows (h = x + residual, its
// squares summed, rstd written) at the memory's rate: 30 us of the 53 us that
// 8192 x 4096 BF16 with residual takes (0.68 of the copy rate over the bytes
// that have to move). The second reads h again, partly from L2 (x and residual
// are read as first to leave it, and its rows go from the last written to the
// first: 70.2 -> 61.2 us at g = 256), and is the block kernel of
// bsgemm_blocks.cuh with y = h * rstd * weight for a value. h takes its usual
// place in L2: stored as last to leave it, it saved 3.5 us in a loop of norms
// alone, nothing where L2 held other data before, and the GEMM behind lost 2 us
// (8192 x 14336 x 4096) to the lines that stayed.
// Slabs of rows with two launches to each cost more than they save (32 MB
// slabs: 58 us). One kernel that holds a row of blocks across a cluster of up to 16
// CTAs, exchanging row sums through distributed shared memory between two
// passes, took 57 us there and 14.7 against 5.4 us on 128 x 7168: its passes
// leave the memory idle at each barrier.
//
// Few rows (a decode step), where launches count: that one kernel, cut down to
// rows that a CTA's threads take at once, with the values held in registers
// between the passes. A row of 7168 BF16 takes 3.7 us: the launch, two trips to
// memory and the cluster's barrier (a second one, which opens the cluster, ends
// under the first loads).

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  void* stream_out;
  uint8_t* q;
  float* scales;
  float* rstd;
  int64_t rows, cols;
  int weight_bf16;
  float eps;
  // few rows only
  int col_blocks;
  int cluster;
  int row_log;      // log2 of the rows a CTA's threads take at once (all of them)
  // many rows only
  int tc_log;       // log2 of the threads to a row
};

__device__ __forceinline__ void load_weight(const void* weight, int is_bf16, int64_t c, float2 (&w)[4]) {
  // (read for every row: kept in L1; not by a read-only load, since the kernel
  // may begin while the one that writes the weight still runs)
  if (is_bf16) {
    Run<true> r;
    r.w[0] = __ldca(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(weight) + c));
    widen<true>(r, w);
  } else {
    Run<false> r;
    r.w[0] = __ldca(reinterpret_cast<const uint4*>(static_cast<const float*>(weight) + c));
    r.w[1] = __ldca(reinterpret_cast<const uint4*>(static_cast<const float*>(weight) + c) + 1);
    widen<false>(r, w);
  }
}

// h = x + residual of a run, rounded to the type. (BF16: the packed addition
// rounds the exact sum once; rounding to FP32 between changes nothing, since a
// sum that needs more than FP32's 24 bits is far from BF16's borders.) It is
// the rounded stream that is normalised: the next layer and the backward pass
// read the same values.
template <bool BF16>
__device__ __forceinline__ Run<BF16> add_runs(const Run<BF16>& x, const Run<BF16>& r) {
  Run<BF16> h;
  if constexpr (BF16) {
    const uint32_t a[4] = {x.w[0].x, x.w[0].y, x.w[0].z, x.w[0].w}, b[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(a[i]), "r"(b[i]));
    h.w[0] = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    float2 v[4], u[4];
    widen<BF16>(x, v);
    widen<BF16>(r, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], u[i]);
    h = narrow<BF16>(v);
  }
  return h;
}

template <bool BF16>
__device__ __forceinline__ float2 add_squares(const Run<BF16>& h, float2 s) {
  float2 v[4];
  widen<BF16>(h, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = bsg::ffma2(v[i], v[i], s);
  return s;
}

__device__ __forceinline__ float rstd_of(const NormParams& p, float sum) {
  return __frsqrt_rn(sum / static_cast<float>(p.cols) + p.eps);
}

// Rows, 2^tc_log threads to each (32 at least): a thread walks its columns,
// four BF16 runs or two FP32 runs in flight.
constexpr int kRowThreads = 256;

template <bool BF16, bool RES>
__global__ void __launch_bounds__(kRowThreads) norm_rows_kernel(const __grid_constant__ NormParams p) {
  constexpr int U = BF16 ? 4 : 2;
  __shared__ float warp_sum[kRowThreads / 32];
  const int tid = threadIdx.x;
  const int tc = 1 << p.tc_log;
  const int t = tid & (tc - 1);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kRowThreads >> p.tc_log) + (tid >> p.tc_log);
  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();
  const bool exists = r < p.rows;
  float2 s = both(0.f);
  if (exists) {
    const int64_t base = r * p.cols;
    const int cols = static_cast<int>(p.cols), stride = tc * kVec;
    int c = t * kVec;
    for (; c + (U - 1) * stride < cols; c += U * stride) {
      Run<BF16> h[U], res[RES ? U : 1];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        h[j] = RES ? load_run_once<BF16>(p.x, base + c + j * stride) : load_run<BF16>(p.x, base + c + j * stride);
        if constexpr (RES) res[j] = load_run_once<BF16>(p.residual, base + c + j * stride);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if constexpr (RES) {
          h[j] = add_runs<BF16>(h[j], res[j]);
          store_run<BF16>(p.stream_out, base + c + j * stride, h[j]);
        }
        s = add_squares<BF16>(h[j], s);
      }
    }
    for (; c < cols; c += stride) {
      Run<BF16> h = RES ? load_run_once<BF16>(p.x, base + c) : load_run<BF16>(p.x, base + c);
      if constexpr (RES) {
        h = add_runs<BF16>(h, load_run_once<BF16>(p.residual, base + c));
        store_run<BF16>(p.stream_out, base + c, h);
      }
      s = add_squares<BF16>(h, s);
    }
  }
  float sum = s.x + s.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tc > 32) {
    if ((tid & 31) == 0) warp_sum[tid / 32] = sum;
    __syncthreads();
    sum = 0.f;
    for (int k = 0; k < tc / 32; ++k) sum += warp_sum[((tid >> p.tc_log) << (p.tc_log - 5)) + k];
  }
  if (exists && t == 0) p.rstd[r] = rstd_of(p, sum);
}

// The block kernel's values: h * rstd * weight.
struct Scaled {
  const float* rstd;
  const void* weight;
  int weight_bf16;
  static constexpr int kInputs = 1;
  static constexpr bool kSums = false;
  template <int NP>
  struct Rows {
    float rs[NP];
  };
  struct Cols {
    float2 w[4];
  };
  template <int NP>
  __device__ __forceinline__ Rows<NP> rows(int64_t row, int left, int step) const {
    Rows<NP> r;
#pragma unroll
    for (int j = 0; j < NP; ++j) r.rs[j] = j * step < left ? __ldcg(rstd + row + j * step) : 0.f;
    return r;
  }
  __device__ __forceinline__ Cols cols(int col, bool exists) const {
    Cols c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = both(0.f);
    if (exists) load_weight(weight, weight_bf16, col, c.w);
    return c;
  }
  template <int NP>
  __device__ __forceinline__ void apply(const Rows<NP>& r, const Cols& c, int j, float2 (&v)[4],
                                        const float2 (&)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(mul2(v[i], both(r.rs[j])), c.w[i]);
  }
};

// Few rows: at most kFewThreads / (g / 8), all in one row of blocks. A cluster
// of C CTAs takes it, 2^row_log rows at once and the threads left over other
// blocks at the same time (`slots` of them): CTA `rank` takes blocks rank + C *
// slot, and so on by C * slots. kFewKeep blocks of a thread stay in registers
// between the passes; where there are more they are read again.
constexpr int kFewThreads = 256;
constexpr int kFewKeep = 4;
constexpr int kMaxCluster = 16;
template <int G>
constexpr int kFewRows = kFewThreads / (G / kVec);

template <int G, bool BF16, int FMT, bool RES>
__global__ void __launch_bounds__(kFewThreads) norm_few_kernel(const __grid_constant__ NormParams p) {
  constexpr int L = G / kVec;          // threads to a row of a block
  constexpr int RP = kFewRows<G>;
  constexpr int K = kFewKeep;
  __shared__ float part[kMaxCluster][RP];  // the row sums of each CTA of the cluster
  __shared__ float own_sum[RP];
  __shared__ float row_rstd[RP];
  __shared__ uint32_t block_max[3][K][RP];

  const int tid = threadIdx.x;
  const int rank = p.cluster > 1 ? static_cast<int>(bsg::cluster_ctarank()) : 0;
  const int rows = static_cast<int>(p.rows);
  const int rp = 1 << p.row_log;
  const int slots = RP >> p.row_log;
  const int col8 = (tid % L) * kVec;
  const int rr = (tid / L) & (rp - 1);
  const int slot = (tid / L) >> p.row_log;
  const int step = p.cluster * slots;      // col_blocks + K * step stays far below 2^31
  const int64_t base = rr * p.cols + col8;

  if (p.cluster > 1) bsg::cluster_open_arrive();
  for (int i = tid; i < 3 * K * RP; i += kFewThreads) (&block_max[0][0][0])[i] = 0;
  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();

  auto inside = [&](int b) {
    return rr < rows && b < p.col_blocks && static_cast<int64_t>(b) * G + col8 < p.cols;
  };
  // ---- pass 1: h and its squares
  Run<BF16> h[K], keep[K];
  float2 ss = both(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) keep[k] = zero_run<BF16>();
  for (int b0 = rank + p.cluster * slot; b0 < p.col_blocks; b0 += K * step) {
    Run<BF16> res[RES ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = b0 + k * step;
      h[k] = zero_run<BF16>();
      if constexpr (RES) res[k] = zero_run<BF16>();
      if (inside(b)) {
        h[k] = load_run<BF16>(p.x, base + static_cast<int64_t>(b) * G);
        if constexpr (RES) res[k] = load_run<BF16>(p.residual, base + static_cast<int64_t>(b) * G);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (RES) {
        const int b = b0 + k * step;
        h[k] = add_runs<BF16>(h[k], res[k]);
        if (inside(b)) store_run<BF16>(p.stream_out, base + static_cast<int64_t>(b) * G, h[k]);
      }
      ss = add_squares<BF16>(h[k], ss);
    }
    if (b0 == rank + p.cluster * slot) {
#pragma unroll
      for (int k = 0; k < K; ++k) keep[k] = h[k];
    }
  }
  float sum = ss.x + ss.y;
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tid % L == 0) own_sum[tid / L] = sum;
  __syncthreads();
  if (p.cluster > 1) bsg::cluster_open_wait();
  if (tid < rows) {
    float s = own_sum[tid];
    for (int k = 1; k < slots; ++k) s += own_sum[k * rp + tid];
    if (p.cluster == 1) {
      part[0][tid] = s;
    } else {
      const uint32_t mine = bsg::smem_addr(&part[rank][tid]);
      for (int d = 0; d < p.cluster; ++d) st_cluster_f32(bsg::mapa_shared(mine, d), s);
    }
  }
  // every thread of the cluster arrives; after it no CTA touches another's
  // shared memory, so any may run on to its exit
  __syncwarp();
  if (p.cluster > 1) bsg::cluster_sync_all();
  else __syncthreads();
  if (tid < rows) {
    float s = part[0][tid];
    for (int k = 1; k < p.cluster; ++k) s += part[k][tid];
    const float v = rstd_of(p, s);
    row_rstd[tid] = v;
    if (rank == 0) p.rstd[tid] = v;
  }
  __syncthreads();

  // ---- pass 2: K blocks of each slot at a time, with one barrier
  const float rs = rr < rows ? row_rstd[rr] : 0.f;
  const void* h_src = RES ? p.stream_out : p.x;
  int buf = 0;
  for (int first = rank; first < p.col_blocks; first += K * step) {
    const int b0 = first + p.cluster * slot;
    float2 v[K][4];
    if (first == rank) {
#pragma unroll
      for (int k = 0; k < K; ++k) h[k] = keep[k];
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        h[k] = zero_run<BF16>();
        if (inside(b0 + k * step)) h[k] = load_run<BF16>(h_src, base + static_cast<int64_t>(b0 + k * step) * G);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = b0 + k * step;
      float2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = both(0.f);
      if (inside(b)) load_weight(p.weight, p.weight_bf16, static_cast<int64_t>(b) * G + col8, w);
      widen<BF16>(h[k], v[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k][i] = mul2(mul2(v[k][i], both(rs)), w[i]);
      // magnitudes are not negative, so their bit patterns order as they do
      float amax = max_abs(0.f, v[k]);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (tid % L == 0) atomicMax(&block_max[buf][k][slot], __float_as_uint(amax));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = b0 + k * step;
      if (b < p.col_blocks) {
        const Scale s = block_scale<FMT>(__uint_as_float(block_max[buf][k][slot]));
        if (rr == 0 && col8 == 0) p.scales[b] = s.s;
        if (inside(b)) store_codes<FMT>(p.q + base + static_cast<int64_t>(b) * G, v[k], s);
      }
    }
    // the maxima of the round before this one: every thread has read them, and
    // they are used again only after the next barrier
    for (int i = tid; i < K * RP; i += kFewThreads) (&block_max[buf == 0 ? 2 : buf - 1][0][0])[i] = 0;
    buf = buf == 2 ? 0 : buf + 1;
  }
}

template <int G, bool BF16, int FMT, bool RES>
bsgemm_status launch_few(NormParams& p, cudaStream_t stream, const bsg_host::DeviceInfo& dev) {
  p.col_blocks = static_cast<int>((p.cols + G - 1) / G);
  p.row_log = 0;
  while ((1 << p.row_log) < p.rows) ++p.row_log;
  // as many CTAs as have blocks for all their slots, at most 16
  p.cluster = 1;
  while (p.cluster < kMaxCluster && p.cluster * (kFewRows<G> >> p.row_log) < p.col_blocks) p.cluster *= 2;
  return launch_rows<norm_few_kernel<G, BF16, FMT, RES>>(dev, p.cluster, kFewThreads, 0, p.cluster, stream, p);
}

template <int G, bool BF16, int FMT>
bsgemm_status few_of(NormParams& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  return p.residual ? launch_few<G, BF16, FMT, true>(p, st, dev) : launch_few<G, BF16, FMT, false>(p, st, dev);
}

template <int G, bool BF16>
bsgemm_status few_of(int fmt, NormParams& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  return fmt == BSGEMM_FP8_E5M2 ? few_of<G, BF16, BSGEMM_FP8_E5M2>(p, st, dev)
                                : few_of<G, BF16, BSGEMM_FP8_E4M3>(p, st, dev);
}

template <bool BF16>
bsgemm_status norm_of(int fmt, int gran, NormParams& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  if (gran == 64 && p.rows <= kFewRows<64>) return few_of<64, BF16>(fmt, p, st, dev);
  if (gran == 128 && p.rows <= kFewRows<128>) return few_of<128, BF16>(fmt, p, st, dev);
  if (gran == 256 && p.rows <= kFewRows<256>) return few_of<256, BF16>(fmt, p, st, dev);
  // threads to a row: 32 where the rows fill the GPU with warps (1024 threads
  // to an SM), else more, as far as there are runs for them
  p.tc_log = 5;
  while ((1 << p.tc_log) < kRowThreads && (kVec << p.tc_log) < p.cols &&
         (p.rows << p.tc_log) < int64_t{dev.num_sms} * 1024)
    ++p.tc_log;
  const int64_t per_cta = kRowThreads >> p.tc_log;
  const int64_t ctas = (p.rows + per_cta - 1) / per_cta;
  bsgemm_status s = p.residual ? launch_rows<norm_rows_kernel<BF16, true>>(dev, ctas, kRowThreads, 0, 1, st, p)
                               : launch_rows<norm_rows_kernel<BF16, false>>(dev, ctas, kRowThreads, 0, 1, st, p);
  if (s != BSGEMM_OK) return s;
  BlockParams b{};
  b.in0 = p.residual ? p.stream_out : p.x;
  b.q = p.q;
  b.scales = p.scales;
  b.rows = p.rows;
  b.cols = p.cols;
  b.backwards = 1;   // the rows written last are the likeliest still in L2
  return launch_blocks<BF16>(gran, fmt, b, Scaled{p.rstd, p.weight, p.weight_bf16}, st, dev);
}

// ------------------------------------------------------------------ backward
//
// A row's gradient needs one sum over its columns (dy * weight * h), so a row
// is read once: a CTA of 256 or 512 threads takes rows of up to 4096 or 8192
// columns, two runs to a thread (256 / TC rows at a time where a row needs only
// TC of them); beyond, a cluster of CTAs takes a row in slices of 8192. Each thread
// keeps the sums of dy * n of its 16 columns over all its rows; at the end they
// are added over the CTA's row groups and written as one row of partial sums,
// and a second kernel adds those rows in order (no atomics: the order never
// changes). B200, BF16 with the skip path's gradient: 8192 x 4096 50.7 us (0.81
// of the copy rate over the bytes that have to move), where a barrier a row and
// the sums at the end show, 32768 x 4096 167 us (0.98). Without the next row's
// runs under way during a row's sum the first took 58.1 us.

constexpr int kBwdMaxThreads = 512;
constexpr int kBwdRuns = 2;          // runs to a thread, TC * 8 columns apart
constexpr int kBwdMaxParts = 640;    // rows of partial sums at most
constexpr int64_t kBwdMaxCols = int64_t{kMaxCluster} * kBwdMaxThreads * kBwdRuns * kVec / 2;   // 65536
template <int T, bool BF16>
constexpr int kBwdCtasPerSm = (BF16 ? 1024 : 512) / T;

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

template <int T, bool BF16, bool SKIP>
__global__ void __launch_bounds__(T, kBwdCtasPerSm<T, BF16>)
    norm_backward_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int V = kBwdRuns;
  constexpr int kWarps = T / 32;
  __shared__ float warp_sum[2][kWarps];
  __shared__ float cta_sum[2][kMaxCluster];   // a cluster's CTAs take one row at a time
  extern __shared__ uint4 fetched[];          // [2][inputs][V][threads] runs: this row's and the next one's
  float2 (&dw_sum)[V * 4][T] = *reinterpret_cast<float2 (*)[V * 4][T]>(fetched);   // at the end

  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int rank = p.cluster > 1 ? static_cast<int>(bsg::cluster_ctarank()) : 0;
  const int part = blockIdx.x / p.cluster;
  const int tc = 1 << p.tc_log;
  const int groups = T >> p.tc_log;
  const int group = tid >> p.tc_log;
  const int group_warps = tc / 32;
  const int run0 = (tid & (tc - 1)) * kVec;   // within the slice; run v is v * tc * 8 on
  const int64_t c0 = static_cast<int64_t>(rank) * p.slice + run0;
  bool in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) in[v] = run0 + v * tc * kVec < p.slice && c0 + v * tc * kVec < p.cols;

  if (p.cluster > 1) bsg::cluster_open_arrive();
  bsg::grid_dependency_wait();

  float2 w[V][4], dw[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[v][i] = dw[v][i] = both(0.f);
    if (in[v]) load_weight(p.weight, p.weight_bf16, c0 + v * tc * kVec, w[v]);
  }
  const float inv_cols = 1.0f / static_cast<float>(p.cols);

  // the part's rows: `groups` at a time, dealt out in turn
  const int64_t stride = static_cast<int64_t>(p.parts) * groups;
  int64_t r = static_cast<int64_t>(part) * groups + group;
  int64_t e = r * p.cols + c0;
  const int64_t e_step = stride * p.cols;
  // A thread's runs of the next row pass through places in shared memory that
  // its warp alone reads (cp.async, two rows' worth), so that loads are in
  // flight through this row's barrier and arithmetic.
  constexpr int kRun = BF16 ? 16 : 32, kElem = BF16 ? 2 : 4, kInputs = SKIP ? 3 : 2;
  // the first column that the thread copies, from its own run's (see fetch_run)
  const int copy = BF16 ? 0 : -(lane * 4);
  bool copied[V], copied2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = run0 + copy + v * tc * kVec, c2 = c + 32 * 4;
    const int64_t slice0 = c0 - run0;
    copied[v] = c < p.slice && slice0 + c < p.cols;
    copied2[v] = c2 < p.slice && slice0 + c2 < p.cols;
  }
  const uint32_t runs = bsg::smem_addr(fetched);
  auto fetch = [&](int64_t row, int64_t at, int to) {
    if (row < p.rows) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (BF16 ? !in[v] : !copied[v]) continue;   // (a second piece lies behind the first)
        const int64_t o = (at + copy + v * tc * kVec) * kElem;
        const char* src[3] = {static_cast<const char*>(p.dy), static_cast<const char*>(p.h),
                              static_cast<const char*>(p.skip)};
#pragma unroll
        for (int k = 0; k < kInputs; ++k)
          fetch_run<BF16, BF16, T, 32>(runs + ((to * kInputs + k) * V + v) * (T * kRun), tid, src[k] + o, true,
                                       copied2[v]);
      }
    }
    fetch_commit();
  };
  auto fetched_of = [&](int from, int input, int v) {
    return fetched_run<BF16, T>(fetched + ((from * kInputs + input) * V + v) * (T * kRun / 16), tid);
  };
  int buf = 0;
  fetch(r, e, 0);
  float rs_next = r < p.rows ? __ldcg(p.rstd + r) : 0.f;
  if (p.cluster > 1) bsg::cluster_open_wait();
  for (int64_t base = static_cast<int64_t>(part) * groups; base < p.rows; base += stride) {
    const bool exists = r < p.rows;
    if constexpr (!BF16) __syncwarp();   // the warp has read the buffer's last row
    fetch(r + stride, e + e_step, buf ^ 1);
    const float rs = rs_next;
    rs_next = r + stride < p.rows ? __ldcg(p.rstd + r + stride) : 0.f;
    fetch_wait<1>();
    if constexpr (!BF16) __syncwarp();   // the warp's other threads' copies
    float2 s2 = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!in[v] || !exists) continue;
      float2 a[4], b[4];
      widen<BF16>(fetched_of(buf, 0, v), a);
      widen<BF16>(fetched_of(buf, 1, v), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 n = mul2(b[i], both(rs));
        dw[v][i] = bsg::ffma2(a[i], n, dw[v][i]);
        s2 = bsg::ffma2(mul2(a[i], w[v][i]), n, s2);
      }
    }
    float s = s2.x + s2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (group_warps > 1 || p.cluster > 1) {
      if (lane == 0) warp_sum[buf][warp] = s;
      __syncthreads();
      // the group's warps, a lane to each: the same order in all of them
      s = warp_sum[buf][(warp & ~(group_warps - 1)) + (lane & (group_warps - 1))];
      for (int o = group_warps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (p.cluster > 1) {
        // (slices of a cluster have more than 4096 columns: one row group)
        if (tid < p.cluster) st_cluster_f32(bsg::mapa_shared(bsg::smem_addr(&cta_sum[buf][rank]), tid), s);
        __syncwarp();
        bsg::cluster_sync_all();
        s = cta_sum[buf][0];
        for (int k = 1; k < p.cluster; ++k) s += cta_sum[buf][k];
      }
    }
    const float m = s * inv_cols;   // mean(dn * n)
    // (the runs are read again rather than held in registers past the barrier)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!in[v] || !exists) continue;
      float2 a[4], b[4];
      widen<BF16>(fetched_of(buf, 0, v), a);
      widen<BF16>(fetched_of(buf, 1, v), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 n = mul2(b[i], both(rs));
        a[i] = mul2(bsg::ffma2(n, both(-m), mul2(a[i], w[v][i])), both(rs));
      }
      if constexpr (SKIP) {
        widen<BF16>(fetched_of(buf, 2, v), b);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = add2(a[i], b[i]);
      }
      store_run<BF16>(p.dx, e + v * tc * kVec, narrow<BF16>(a));
    }
    r += stride;
    e += e_step;
    // the sums are double-buffered: a thread writes a buffer again two rows
    // on, past a barrier that follows every read of it
    buf ^= 1;
  }

  // The next kernel may start now, not before: this one fills every SM, and a
  // kernel that settled beside its last CTAs to come would keep them waiting
  // (61 against 51 us on 8192 x 4096 BF16).
  bsg::grid_launch_dependents();
  // the row groups' sums, added in order by the first group's threads (in the
  // fetched runs' place: none is in flight, and all have been read)
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw_sum[v * 4 + i][tid] = dw[v][i];
  __syncthreads();
  if (group == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[v][i] = add2(dw[v][i], dw_sum[v * 4 + i][(g << p.tc_log) + tid]);
      if (in[v])
        store_run<false>(p.part, static_cast<int64_t>(part) * p.cols + c0 + v * tc * kVec, narrow<false>(dw[v]));
    }
  }
}

// One CTA adds 32 columns: 32 warps take every 32nd row, then one warp adds
// the 32 sums in order. The loads of kSumRows rows are in flight at once (20 of
// them took 52 registers, which kept the CTAs out until the last kernel's had
// left: 333 x 1552 7.1 against 5.2 us).
constexpr int kSumRows = 5;
__global__ void __launch_bounds__(1024, 2) column_sum_kernel(const float* part, int parts, int64_t cols, float* out) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  bsg::grid_dependency_wait();
  float s = 0.f;
  if (c < cols) {
    for (int i = warp; i < parts; i += 32 * kSumRows) {
      float v[kSumRows];
#pragma unroll
      for (int k = 0; k < kSumRows; ++k)
        v[k] = i + 32 * k < parts ? __ldcg(part + static_cast<int64_t>(i + 32 * k) * cols + c) : 0.f;
#pragma unroll
      for (int k = 0; k < kSumRows; ++k) s += v[k];
    }
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
bsgemm_status launch_column_sum(const float* part, int parts, int64_t cols, float* out, cudaStream_t stream,
                                const bsg_host::DeviceInfo& dev) {
  return launch_rows<bsgn::column_sum_kernel>(dev, (cols + 31) / 32, 1024, 0, 1, stream, part, parts, cols, out);
}
}  // namespace bsgr

extern "C" bsgemm_status bsgemm_rms_norm_quantize_fp8(int src_dtype, int weight_dtype, int fp8_format,
                                                      const void* x, const void* residual, const void* weight,
                                                      float eps, int64_t rows, int64_t cols, int gran,
                                                      void* residual_out, void* q, float* scales, float* rstd,
                                                      bsgemm_stream_t stream) {
  if (!x || !weight || !q || !scales || !rstd || (residual != nullptr) != (residual_out != nullptr))
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
  return src_dtype == BSGEMM_SRC_BF16 ? bsgn::norm_of<true>(fp8_format, gran, p, s, dev)
                                      : bsgn::norm_of<false>(fp8_format, gran, p, s, dev);
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
  const int64_t span = bsgn::kBwdRuns * bsgr::kVec;   // columns to a thread
  const int threads = cols <= 256 * span ? 256 : 512;
  p.cluster = 1;
  while (int64_t{p.cluster} * threads * span < cols) p.cluster *= 2;
  const int64_t runs = cols / bsgr::kVec;
  p.slice = static_cast<int>((runs + p.cluster - 1) / p.cluster * bsgr::kVec);
  p.tc_log = 5;
  while ((span << p.tc_log) < p.slice) ++p.tc_log;
  const int64_t batch = threads >> p.tc_log;
  const int64_t batches = (rows + batch - 1) / batch;
  int64_t parts = int64_t{dev.num_sms} * ((bf16 ? 1024 : 512) / threads) / p.cluster;
  if (parts < 1) parts = 1;
  if (parts > batches) parts = batches;
  if (parts > bsgn::kBwdMaxParts) parts = bsgn::kBwdMaxParts;
  p.parts = static_cast<int>(parts);
  // one row of partial sums is the result itself
  p.part = parts == 1 ? dweight : static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t grid = parts * p.cluster;
#define BSGN_GO(T, BF, SK)                                                                                    \
  bsgr::launch_rows<bsgn::norm_backward_kernel<T, BF, SK>>(                                                   \
      dev, grid, T, 2 * (SK ? 3 : 2) * bsgn::kBwdRuns * T * (BF ? 16 : 32), p.cluster, s, p)
  if (threads == 256) {
    if (bf16) st = skip ? BSGN_GO(256, true, true) : BSGN_GO(256, true, false);
    else      st = skip ? BSGN_GO(256, false, true) : BSGN_GO(256, false, false);
  } else {
    if (bf16) st = skip ? BSGN_GO(512, true, true) : BSGN_GO(512, true, false);
    else      st = skip ? BSGN_GO(512, false, true) : BSGN_GO(512, false, false);
  }
#undef BSGN_GO
  if (st != BSGEMM_OK || parts == 1) return st;
  return bsgr::launch_column_sum(p.part, p.parts, cols, dweight, s, dev);
}

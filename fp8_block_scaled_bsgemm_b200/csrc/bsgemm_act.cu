// Activations in front of the quantiser, and the gradient of the GEMM's
// epilogue.
//
// Forward:   q, s of act(z), z the product with its bias as the GEMM stored it
//            (kept for the backward pass), so the activation's own tensor is
//            never written.
// Backward:  for out = act(z) + residual, z = acc + bias, and the gradient dout
//            of out:  dz = dout * act'(z)  as codes and scales (the operand of
//            the two gradient products), dbias[n] = sum over rows of dz.
//            The residual's gradient is dout itself.
// Per g x g block, as in the quantiser: s = amax / FMAX (1 if that is 0),
// q = FP8 code of value / s.
//
// One CTA per block with g <= 128; a cluster of four per block with g = 256,
// 64 of its rows each. A thread computes its values once, keeps them in
// registers past the block's amax, and encodes them.
#include "bsgemm_host.h"
#include "bsgemm_rows.cuh"

namespace bsga {

using namespace bsgr;

enum { kNone = BSGEMM_ACT_NONE, kRelu = BSGEMM_ACT_RELU, kGelu = BSGEMM_ACT_GELU };

// The normal distribution function and density of two values.
//
// For u = |z| and t = 1 / (1 + p u), Phi(-u) = exp(-u^2 / 2) * Q(t): the factor
// beside the exponential is smooth and monotonic in u, and a polynomial in t
// without a constant term follows it over all of [0, inf). The coefficients
// are an iteratively reweighted least-squares fit (Lawson's method) of degree
// 9 at 3000 Chebyshev nodes of t, u up to 40: relative error 9e-8 at most.
// With FP32's own roundings Phi is within 1.9e-7 everywhere (400001 points of
// u in [0, 40]), and its lower tail within 7e-7 of itself for u < 3 (1 + erf
// loses that tail to cancellation). One exponential and one reciprocal serve both results, and
// the polynomial runs two values to an instruction; with erff and expf apart
// the arithmetic would take longer than the memory traffic.
constexpr float kP = 0.36f;

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ void normal2(float2 z, float2& cdf, float2& pdf) {
  const float2 u = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 d = bsg::ffma2(u, both(kP), both(1.0f));
  const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  float2 q = both(-0.030238333f);
  q = bsg::ffma2(q, t, both(0.13950870f));
  q = bsg::ffma2(q, t, both(-0.22360013f));
  q = bsg::ffma2(q, t, both(0.10736972f));
  q = bsg::ffma2(q, t, both(-0.00038668368f));
  q = bsg::ffma2(q, t, both(0.09603746f));
  q = bsg::ffma2(q, t, both(0.12400974f));
  q = bsg::ffma2(q, t, both(0.14368188f));
  q = bsg::ffma2(q, t, both(0.14361767f));
  q = mul2(q, t);
  // exp(-z^2 / 2) = 2^(-z^2 log2(e) / 2)
  const float2 a = mul2(mul2(z, z), both(-0.72134752f));
  const float2 e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
  const float2 tail = mul2(e, q);
  cdf = make_float2(z.x < 0.f ? tail.x : 1.0f - tail.x, z.y < 0.f ? tail.y : 1.0f - tail.y);
  pdf = mul2(e, both(0.39894228f));
}

template <int ACT>
__device__ __forceinline__ float2 act2(float2 z) {
  if constexpr (ACT == kRelu) return make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f));
  if constexpr (ACT == kGelu) {
    float2 cdf, pdf;
    normal2(z, cdf, pdf);
    return mul2(z, cdf);
  }
  return z;
}

// d * act'(z); ReLU's slope at 0 is 0
template <int ACT>
__device__ __forceinline__ float2 slope2(float2 d, float2 z) {
  if constexpr (ACT == kRelu) return make_float2(z.x > 0.f ? d.x : 0.f, z.y > 0.f ? d.y : 0.f);
  if constexpr (ACT == kGelu) {
    float2 cdf, pdf;
    normal2(z, cdf, pdf);
    return mul2(d, bsg::ffma2(z, pdf, cdf));
  }
  return d;
}

template <int G>
constexpr int kParts = G == 256 ? 4 : 1;   // CTAs to a block
template <int G>
constexpr int kThreads = G == 64 ? 256 : 512;

struct Params {
  const void* z;       // null where the activation is none
  const void* dout;    // backward only
  uint8_t* q;
  float* scales;
  float* part;         // backward: column sums of each CTA's rows, or null
  int64_t rows, cols;
  int col_blocks;
};

template <int G, bool BF16, int FMT, int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads<G>, kThreads<G> == 256 ? 4 : 2)
    act_quant_kernel(const __grid_constant__ Params p) {
  constexpr int T = kThreads<G>;
  constexpr int P = kParts<G>;
  constexpr int L = G / kVec;          // threads to a row
  constexpr int RP = T / L;            // rows at a time
  constexpr int NP = G / P / RP;       // rows a thread holds
  constexpr int W = T / 32;
  static_assert(NP * RP * P == G, "the rows of a block are dealt out evenly");
  __shared__ float warp_max[W];
  __shared__ float part_max[P];
  __shared__ float col_sum[BWD ? W : 1][BWD ? G : 1];

  const int tid = threadIdx.x;
  const int64_t blk = blockIdx.x / P;
  const int part = static_cast<int>(blockIdx.x % P);   // the CTA's rank in its cluster
  const int64_t rb = blk / p.col_blocks;
  const int64_t c0 = (blk - rb * p.col_blocks) * G;
  const int64_t r0 = rb * G + part * (G / P) + tid / L;
  const int col8 = (tid % L) * kVec;
  const int64_t c = c0 + col8;
  const bool in = c < p.cols;

  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();

  Run<BF16> a[NP], b[BWD && ACT != kNone ? NP : 1];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int64_t r = r0 + j * RP;
    const bool ok = in && r < p.rows;
    a[j] = zero_run<BF16>();
    if (ok) a[j] = load_run<BF16>(BWD ? p.dout : p.z, r * p.cols + c);
    if constexpr (BWD && ACT != kNone) {
      b[j] = zero_run<BF16>();
      if (ok) b[j] = load_run<BF16>(p.z, r * p.cols + c);
    }
  }
  // values outside the matrix are 0: act(0) = 0, and 0 * act'(0) = 0
  float2 v[NP][4];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    widen<BF16>(a[j], v[j]);
    if constexpr (BWD && ACT != kNone) {
      float2 z[4];
      widen<BF16>(b[j], z);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = slope2<ACT>(v[j][i], z[i]);
    } else if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = act2<ACT>(v[j][i]);
    }
    amax = max_abs(amax, v[j]);
  }
  // magnitudes are not negative, so their bit patterns order as they do
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((tid & 31) == 0) warp_max[tid / 32] = amax;
  if constexpr (BWD) {
    if (p.part != nullptr) {
      // the thread's rows, then the warp's (32 / L of them hold the same columns)
      float2 s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = v[0][i];
#pragma unroll
        for (int j = 1; j < NP; ++j) s[i] = add2(s[i], v[j][i]);
#pragma unroll
        for (int o = L; o < 32; o *= 2) {
          s[i].x += __shfl_xor_sync(0xffffffffu, s[i].x, o);
          s[i].y += __shfl_xor_sync(0xffffffffu, s[i].y, o);
        }
        if ((tid & 31) < L) *reinterpret_cast<float2*>(&col_sum[tid / 32][col8 + 2 * i]) = s[i];
      }
    }
  }
  __syncthreads();
  amax = warp_max[0];
#pragma unroll
  for (int w = 1; w < W; ++w) amax = fmaxf(amax, warp_max[w]);
  if constexpr (P > 1) {
    // each CTA writes its share of the amax into every CTA of the cluster; no
    // CTA touches another's shared memory after the barrier
    if (tid < P) st_cluster_f32(bsg::mapa_shared(bsg::smem_addr(&part_max[part]), tid), amax);
    __syncwarp();
    bsg::cluster_sync_all();
#pragma unroll
    for (int k = 0; k < P; ++k) amax = fmaxf(amax, part_max[k]);
  }
  const float s = block_scale<FMT>(amax);
  const float rcp = __frcp_rn(s);
  if (tid == 0 && part == 0) p.scales[blk] = s;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int64_t r = r0 + j * RP;
    if (in && r < p.rows) store_codes<FMT>(p.q, r * p.cols + c, v[j], s, rcp);
  }
  if constexpr (BWD) {
    if (p.part != nullptr && tid < G && c0 + tid < p.cols) {
      float sum = col_sum[0][tid];
#pragma unroll
      for (int w = 1; w < W; ++w) sum += col_sum[w][tid];
      p.part[(rb * P + part) * p.cols + c0 + tid] = sum;
    }
  }
}

// Rows of partial column sums of a backward call.
inline int64_t parts_of(int64_t rows, int gran) { return (rows + gran - 1) / gran * (gran == 256 ? 4 : 1); }

template <int G, bool BF16, int FMT, int ACT, bool BWD>
bsgemm_status launch(const Params& p, cudaStream_t stream) {
  const int64_t blocks = (p.rows + G - 1) / G * p.col_blocks;
  return launch_rows(act_quant_kernel<G, BF16, FMT, ACT, BWD>, blocks * kParts<G>, kThreads<G>, 0, kParts<G>,
                     stream, p);
}

template <int G, bool BF16, int FMT, bool BWD>
bsgemm_status act_of(int act, Params& p, cudaStream_t st) {
  p.col_blocks = static_cast<int>((p.cols + G - 1) / G);
  if (act == kGelu) return launch<G, BF16, FMT, kGelu, BWD>(p, st);
  if (act == kRelu) return launch<G, BF16, FMT, kRelu, BWD>(p, st);
  // forward without an activation is the quantiser's own call
  if constexpr (BWD) return launch<G, BF16, FMT, kNone, BWD>(p, st);
  return BSGEMM_ERR_INVALID_ARG;
}

template <bool BWD>
bsgemm_status run(int src, int fmt, int act, int gran, Params& p, cudaStream_t st) {
  const bool bf16 = src == BSGEMM_SRC_BF16, e5 = fmt == BSGEMM_FP8_E5M2;
#define BSGA_GO(G)                                                                                      \
  if (bf16) return e5 ? act_of<G, true, BSGEMM_FP8_E5M2, BWD>(act, p, st)                              \
                      : act_of<G, true, BSGEMM_FP8_E4M3, BWD>(act, p, st);                             \
  return e5 ? act_of<G, false, BSGEMM_FP8_E5M2, BWD>(act, p, st) : act_of<G, false, BSGEMM_FP8_E4M3, BWD>(act, p, st)
  switch (gran) {
    case 64:  BSGA_GO(64);
    case 128: BSGA_GO(128);
    default:  BSGA_GO(256);
  }
#undef BSGA_GO
}

// Outputs may share no memory with each other or with the inputs.
bool overlapping(int src_dtype, int64_t rows, int64_t cols, int gran, const void* z, const void* dout, const void* q,
                 const void* scales, const void* dbias, const void* workspace, size_t workspace_bytes) {
  const size_t n = static_cast<size_t>(rows) * static_cast<size_t>(cols);
  const size_t bytes = n * (src_dtype == BSGEMM_SRC_BF16 ? 2 : 4);
  const Span out[] = {{q, n}, {scales, blocks_bytes(rows, cols, gran)},
                      {dbias, static_cast<size_t>(cols) * sizeof(float)}, {workspace, workspace_bytes}};
  const Span in[] = {{z, bytes}, {dout, bytes}};
  return any_overlap(out, in);
}

bsgemm_status check(int src_dtype, int fp8_format, int activation, int64_t rows, int64_t cols, int gran) {
  if (fp8_format != BSGEMM_FP8_E4M3 && fp8_format != BSGEMM_FP8_E5M2) return BSGEMM_ERR_INVALID_ARG;
  if (activation < BSGEMM_ACT_NONE || activation > BSGEMM_ACT_GELU) return BSGEMM_ERR_INVALID_ARG;
  if (gran != 64 && gran != 128 && gran != 256) return BSGEMM_ERR_UNSUPPORTED_GRAN;
  return check_rows(src_dtype, rows, cols);
}

}  // namespace bsga

extern "C" bsgemm_status bsgemm_activation_quantize_fp8(int src_dtype, int fp8_format, int activation, const void* z,
                                                        int64_t rows, int64_t cols, int gran, void* q, float* scales,
                                                        bsgemm_stream_t stream) {
  if (!z || !q || !scales || activation == BSGEMM_ACT_NONE) return BSGEMM_ERR_INVALID_ARG;
  bsgemm_status st = bsga::check(src_dtype, fp8_format, activation, rows, cols, gran);
  if (st != BSGEMM_OK) return st;
  if (!bsgr::aligned(z, 16) || !bsgr::aligned(q, 16) || !bsgr::aligned(scales, 4)) return BSGEMM_ERR_MISALIGNED;
  if (bsga::overlapping(src_dtype, rows, cols, gran, z, nullptr, q, scales, nullptr, nullptr, 0))
    return BSGEMM_ERR_INVALID_ARG;
  bsg_host::DeviceInfo dev;
  st = bsg_host::device_info(dev);
  if (st != BSGEMM_OK) return st;
  bsga::Params p{};
  p.z = z;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.rows = rows;
  p.cols = cols;
  return bsga::run<false>(src_dtype, fp8_format, activation, gran, p, static_cast<cudaStream_t>(stream));
}

extern "C" size_t bsgemm_activation_backward_workspace(int64_t rows, int64_t cols, int gran) {
  if (rows <= 0 || cols <= 0 || (gran != 64 && gran != 128 && gran != 256)) return 0;
  const int64_t parts = bsga::parts_of(rows, gran);
  return parts == 1 ? 0 : static_cast<size_t>(parts) * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" bsgemm_status bsgemm_activation_backward_quantize_fp8(int src_dtype, int fp8_format, int activation,
                                                                 const void* dout, const void* z, int64_t rows,
                                                                 int64_t cols, int gran, void* q, float* scales,
                                                                 float* dbias, void* workspace,
                                                                 size_t workspace_bytes, bsgemm_stream_t stream) {
  if (!dout || !q || !scales) return BSGEMM_ERR_INVALID_ARG;
  bsgemm_status st = bsga::check(src_dtype, fp8_format, activation, rows, cols, gran);
  if (st != BSGEMM_OK) return st;
  if ((z != nullptr) != (activation != BSGEMM_ACT_NONE)) return BSGEMM_ERR_INVALID_ARG;
  const size_t need = dbias ? bsgemm_activation_backward_workspace(rows, cols, gran) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return BSGEMM_ERR_INVALID_ARG;
  if (!bsgr::aligned(dout, 16) || !bsgr::aligned(z, 16) || !bsgr::aligned(q, 16) || !bsgr::aligned(scales, 4) ||
      !bsgr::aligned(dbias, 4) || !bsgr::aligned(workspace, 4))
    return BSGEMM_ERR_MISALIGNED;
  if (bsga::overlapping(src_dtype, rows, cols, gran, z, dout, q, scales, dbias, need > 0 ? workspace : nullptr, need))
    return BSGEMM_ERR_INVALID_ARG;
  bsg_host::DeviceInfo dev;
  st = bsg_host::device_info(dev);
  if (st != BSGEMM_OK) return st;
  bsga::Params p{};
  p.z = z;
  p.dout = dout;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.part = need > 0 ? static_cast<float*>(workspace) : dbias;   // one row of sums is the result itself
  p.rows = rows;
  p.cols = cols;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = bsga::run<true>(src_dtype, fp8_format, activation, gran, p, s);
  if (st != BSGEMM_OK || need == 0) return st;
  return bsgr::launch_column_sum(p.part, static_cast<int>(bsga::parts_of(rows, gran)), cols, dbias, s);
}

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
// One CTA takes a block with g <= 128; a cluster of four one with g = 256, 64 of
// its rows each. A thread computes its values once, keeps them in registers
// past the block's amax, and encodes them.
#include "bsgemm_host.h"
#include "bsgemm_rows.cuh"

namespace bsga {

using namespace bsgr;

enum { kNone = BSGEMM_ACT_NONE, kRelu = BSGEMM_ACT_RELU, kGelu = BSGEMM_ACT_GELU };

// GELU and its slope, eight values (a run) at a time.
//
// With u = |z| and the lower tail of the normal distribution T = Phi(-u),
//   z Phi(z)          = max(z, 0) - u T,
//   Phi(z) + z phi(z) = 1/2 + sign(z) (1/2 - T + u phi(u)).
// log2 T is smooth and nearly quadratic in u, so T = 2^P(u) with a polynomial P
// of degree 6: one exponential and no division or case distinction. P is an
// iteratively reweighted least-squares fit (Lawson's method, 6000 Chebyshev
// nodes of [0, 6.5]) that weights the error by T, so T is off by 1.1e-7 at most,
// and falls below 2^-126 before u = 14, where u is clamped. With FP32's
// roundings GELU is within 2e-7 |z| and the slope within 3e-7 over 2.8 million
// points of [-14, 14]: what 1 + erf gives in FP32.
// Arithmetic, not memory, bounded these kernels at first. On 8192 x 14336 BF16:
// erff alone 30 instructions a value; exp(-u^2/2) times a polynomial of 1 / (1 +
// p u) 110 us (two special-function results a value are 53 us by themselves);
// exp(-u^2/2) times a polynomial of degree 10 in u 94 us.
// The steps of the polynomial run over the run's four pairs side by side: a
// packed instruction takes its constant from a register pair, which is then
// built once per step rather than once per pair and step.
constexpr float kUMax = 14.0f;

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 exp2_approx(float2 v) { return make_float2(exp2_approx(v.x), exp2_approx(v.y)); }

// n = -min(|z|, 14) and T = Phi(n)
__device__ __forceinline__ void normal_tail(const float2 (&z)[4], float2 (&n)[4], float2 (&t)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = make_float2(fmaxf(-fabsf(z[i].x), -kUMax), fmaxf(-fabsf(z[i].y), -kUMax));
    t[i] = both(1.91764611e-5f);
  }
  const float coef[6] = {6.58616424e-4f, 7.75443763e-3f, 5.2965425e-2f, -0.459060252f, 1.15112209f, -0.999999702f};
#pragma unroll
  for (int k = 0; k < 6; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = bsg::ffma2(t[i], n[i], both(coef[k]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = exp2_approx(t[i]);
}

template <int ACT>
__device__ __forceinline__ void act_run(float2 (&z)[4]) {
  float2 n[4], t[4];
  if constexpr (ACT == kGelu) normal_tail(z, n, t);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[i] = make_float2(fmaxf(z[i].x, 0.f), fmaxf(z[i].y, 0.f));
    if constexpr (ACT == kGelu) z[i] = bsg::ffma2(n[i], t[i], z[i]);
  }
}

// d * act'(z); ReLU's slope at 0 is 0
template <int ACT>
__device__ __forceinline__ void slope_run(float2 (&d)[4], const float2 (&z)[4]) {
  float2 n[4], t[4];
  if constexpr (ACT == kGelu) normal_tail(z, n, t);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ACT == kRelu) d[i] = make_float2(z[i].x > 0.f ? d[i].x : 0.f, z[i].y > 0.f ? d[i].y : 0.f);
    if constexpr (ACT == kGelu) {
      // phi(u) = 2^(-u^2 log2(e) / 2 - log2(2 pi) / 2); h = T - 1/2 - u phi(u)
      const float2 phi = exp2_approx(bsg::ffma2(mul2(n[i], n[i]), both(-0.72134752f), both(-1.32574807f)));
      float2 h = bsg::ffma2(n[i], phi, add2(t[i], both(-0.5f)));
      // -h times the sign of z (h may be of either sign itself)
      h.x = __uint_as_float(__float_as_uint(h.x) ^ (~__float_as_uint(z[i].x) & 0x80000000u));
      h.y = __uint_as_float(__float_as_uint(h.y) ^ (~__float_as_uint(z[i].y) & 0x80000000u));
      d[i] = mul2(d[i], add2(h, both(0.5f)));
    }
  }
}

template <int G>
constexpr int kParts = G == 256 ? 4 : 1;   // CTAs to a block
template <int G>
constexpr int kThreads = G == 64 ? 256 : 512;
template <int G>
constexpr int kCtasPerSm = G == 64 ? 4 : 2;

// A thread's runs of a block pass through shared memory (cp.async into places
// that this thread alone reads, so no barrier is needed), which keeps the next
// block's loads in flight while this one is computed without holding them in
// registers. Two buffers where they fit beside a second CTA, else one, refilled
// once the block's values are in registers; none for the widest case.
template <int G, bool BF16, bool IN2>
constexpr int kBufBytes = kThreads<G> * (G / kParts<G> / (kThreads<G> / (G / kVec))) * (BF16 ? 16 : 32) * (IN2 ? 2 : 1);
template <int G, bool BF16, bool IN2>
constexpr int kBufs = kBufBytes<G, BF16, IN2> * kCtasPerSm<G> * 2 <= 192 * 1024 ? 2
                      : kBufBytes<G, BF16, IN2> * kCtasPerSm<G> <= 192 * 1024 ? 1 : 0;

struct Params {
  const void* z;       // null where the activation is none
  const void* dout;    // backward only
  uint8_t* q;
  float* scales;
  float* part;         // backward: column sums of each CTA's rows, or null
  int64_t rows, cols;
  int row_blocks, col_blocks;
  int step_rb, step_cb;   // from a CTA's block to its next: rows and columns of blocks
};

// A walk over the matrix's blocks in row-major order, without divisions.
struct Walk {
  int rb, cb;
  __device__ __forceinline__ void next(const Params& p) {
    rb += p.step_rb;
    cb += p.step_cb;
    if (cb >= p.col_blocks) {
      cb -= p.col_blocks;
      ++rb;
    }
  }
};

// Copies a run into shared memory, zeros (and no access) where it lies outside
// the matrix.
template <bool BF16>
__device__ __forceinline__ void fetch_run(uint32_t dst, const char* src, bool in) {
  const int bytes = in ? 16 : 0;
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * h), "l"(src + 16 * h), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Persistent: CTA (or cluster) k takes blocks k, k + grid, ... in row-major
// order.
template <int G, bool BF16, int FMT, int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads<G>, kCtasPerSm<G>) act_quant_kernel(const __grid_constant__ Params p) {
  constexpr int T = kThreads<G>;
  constexpr int P = kParts<G>;
  constexpr int L = G / kVec;          // threads to a row
  constexpr int RP = T / L;            // rows at a time
  constexpr int NP = G / P / RP;       // rows a thread holds
  constexpr int W = T / 32;
  constexpr bool IN2 = BWD && ACT != kNone;   // two inputs: dout and z
  constexpr int kBuf = kBufs<G, BF16, IN2>;
  constexpr int kRun = BF16 ? 16 : 32;
  static_assert(NP * RP * P == G, "the rows of a block are dealt out evenly");
  extern __shared__ uint4 fetched[];   // [kBuf][inputs][NP][T] runs
  __shared__ float warp_max[2][W];
  __shared__ float part_max[2][P];
  __shared__ float col_sum[BWD ? 2 : 1][BWD ? W : 1][BWD ? G : 1];

  constexpr int kElem = BF16 ? 2 : 4;
  const int tid = threadIdx.x;
  const int part = static_cast<int>(blockIdx.x % P);   // the CTA's rank in its cluster
  const int row0 = part * (G / P) + tid / L;           // the thread's first row of a block
  const int col8 = (tid % L) * kVec;
  const int64_t row_step = RP * p.cols;                // elements from one of the thread's rows to the next
  const int cols = static_cast<int>(p.cols);           // at most 2^30
  const int rows = static_cast<int>(p.rows);

  // the thread's first element in block w, and how many of its NP rows exist
  auto place = [&](const Walk& w, int64_t& at) {
    at = (static_cast<int64_t>(w.rb) * G + row0) * p.cols + static_cast<int64_t>(w.cb) * G + col8;
    const int left = rows - w.rb * G - row0;           // rows + G stays below 2^31
    return w.cb * G + col8 < cols ? left : 0;          // row j * RP of the thread exists if below this
  };

  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();

  const uint32_t own = kBuf > 0 ? bsg::smem_addr(fetched) + tid * kRun : 0;
  auto slot = [&](int buf, int input, int j) -> uint32_t {
    return own + ((buf * (IN2 ? 2 : 1) + input) * NP + j) * (T * kRun);
  };
  const char* in0 = static_cast<const char*>(BWD ? p.dout : p.z);
  const char* in1 = static_cast<const char*>(p.z);
  auto fetch = [&](const Walk& w, int buf) {
    if (w.rb < p.row_blocks) {
      int64_t at;
      const int left = place(w, at);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const bool in = j * RP < left;
        const int64_t e = in ? (at + j * row_step) * kElem : 0;
        fetch_run<BF16>(slot(buf, 0, j), in0 + e, in);
        if constexpr (IN2) fetch_run<BF16>(slot(buf, 1, j), in1 + e, in);
      }
    }
    fetch_commit();
  };
  auto fetched_run = [&](int buf, int input, int j) {
    Run<BF16> r;
    const uint4* at = fetched + (((buf * (IN2 ? 2 : 1) + input) * NP + j) * T + tid) * (kRun / 16);
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = at[h];
    return r;
  };

  Walk w{static_cast<int>(blockIdx.x / P) / p.col_blocks, static_cast<int>(blockIdx.x / P) % p.col_blocks};
  if constexpr (kBuf > 0) fetch(w, 0);
  int par = 0;   // parity of the block: which copy of the exchanged values it uses
  for (; w.rb < p.row_blocks; par ^= 1) {
    int64_t at;
    const int left = place(w, at);
    const int64_t blk = static_cast<int64_t>(w.rb) * p.col_blocks + w.cb;
    const int c0 = w.cb * G;
    const int64_t part_row = static_cast<int64_t>(w.rb) * P + part;
    w.next(p);
    const int buf = kBuf == 2 ? par : 0;
    if constexpr (kBuf == 2) {
      fetch(w, par ^ 1);
      fetch_wait<1>();
    } else if constexpr (kBuf == 1) {
      fetch_wait<0>();
    }
    // values outside the matrix are 0: act(0) = 0, and 0 * act'(0) = 0
    float2 v[NP][4];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      Run<BF16> a, b;
      if constexpr (kBuf > 0) {
        a = fetched_run(buf, 0, j);
        if constexpr (IN2) b = fetched_run(buf, 1, j);
      } else {
        a = b = zero_run<BF16>();
        if (j * RP < left) {
          a = load_run<BF16>(in0, at + j * row_step);
          if constexpr (IN2) b = load_run<BF16>(in1, at + j * row_step);
        }
      }
      widen<BF16>(a, v[j]);
      if constexpr (IN2) {
        float2 z[4];
        widen<BF16>(b, z);
        slope_run<ACT>(v[j], z);
      } else if constexpr (!BWD) {
        act_run<ACT>(v[j]);
      }
      amax = max_abs(amax, v[j]);
    }
    // magnitudes are not negative, so their bit patterns order as they do
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if ((tid & 31) == 0) warp_max[par][tid / 32] = amax;
    if constexpr (BWD) {
      if (p.part != nullptr) {
        // the thread's rows, then the warp's (32 / L of them hold the same columns)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 s = v[0][i];
#pragma unroll
          for (int j = 1; j < NP; ++j) s = add2(s, v[j][i]);
#pragma unroll
          for (int o = L; o < 32; o *= 2) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
          }
          if ((tid & 31) < L) *reinterpret_cast<float2*>(&col_sum[par][tid / 32][col8 + 2 * i]) = s;
        }
      }
    }
    // (a copy of the exchanged values is written again two blocks on, past a
    // barrier that follows every read of it)
    __syncthreads();
    // past the barrier every value of the block is in a register
    if constexpr (kBuf == 1) fetch(w, 0);
    static_assert(W <= 32, "one value a lane");
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(warp_max[par][(tid & 31) % W])));
    if constexpr (P > 1) {
      // each CTA writes its share of the amax into every CTA of the cluster
      if (tid < P) st_cluster_f32(bsg::mapa_shared(bsg::smem_addr(&part_max[par][part]), tid), amax);
      __syncwarp();
      bsg::cluster_sync_all();
#pragma unroll
      for (int k = 0; k < P; ++k) amax = fmaxf(amax, part_max[par][k]);
    }
    const Scale s = block_scale<FMT>(amax);
    if (tid == 0 && part == 0) p.scales[blk] = s.s;
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if (j * RP < left) store_codes<FMT>(p.q + at + j * row_step, v[j], s);
    if constexpr (BWD) {
      if (p.part != nullptr && tid < G && c0 + tid < cols) {
        float sum = col_sum[par][0][tid];
#pragma unroll
        for (int k = 1; k < W; ++k) sum += col_sum[par][k][tid];
        p.part[part_row * p.cols + c0 + tid] = sum;
      }
    }
  }
  // no copy is in flight here: fetches past the last block are empty, and the
  // last block's were waited for
}

// Rows of partial column sums of a backward call.
inline int64_t parts_of(int64_t rows, int gran) { return (rows + gran - 1) / gran * (gran == 256 ? 4 : 1); }

template <int G, bool BF16, int FMT, int ACT, bool BWD>
bsgemm_status launch(Params& p, cudaStream_t stream, const bsg_host::DeviceInfo& dev) {
  constexpr bool IN2 = BWD && ACT != kNone;
  constexpr int kSmem = kBufBytes<G, BF16, IN2> * kBufs<G, BF16, IN2>;
  auto kern = act_quant_kernel<G, BF16, FMT, ACT, BWD>;
  static bsg_host::PerDeviceOnce setup;
  if (!setup.done(dev.ordinal)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return BSGEMM_ERR_CUDA;
    setup.mark(dev.ordinal);
  }
  p.row_blocks = static_cast<int>((p.rows + G - 1) / G);
  int64_t units = int64_t{dev.num_sms} * kCtasPerSm<G> / kParts<G>;   // blocks taken at the same time
  const int64_t blocks = static_cast<int64_t>(p.row_blocks) * p.col_blocks;
  if (units > blocks) units = blocks;
  p.step_rb = static_cast<int>(units / p.col_blocks);
  p.step_cb = static_cast<int>(units % p.col_blocks);
  return launch_rows(kern, units * kParts<G>, kThreads<G>, kSmem, kParts<G>, stream, p);
}

template <int G, bool BF16, int FMT, bool BWD>
bsgemm_status act_of(int act, Params& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  p.col_blocks = static_cast<int>((p.cols + G - 1) / G);
  if (act == kGelu) return launch<G, BF16, FMT, kGelu, BWD>(p, st, dev);
  if (act == kRelu) return launch<G, BF16, FMT, kRelu, BWD>(p, st, dev);
  // forward without an activation is the quantiser's own call
  if constexpr (BWD) return launch<G, BF16, FMT, kNone, BWD>(p, st, dev);
  return BSGEMM_ERR_INVALID_ARG;
}

template <bool BWD>
bsgemm_status run(int src, int fmt, int act, int gran, Params& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  const bool bf16 = src == BSGEMM_SRC_BF16, e5 = fmt == BSGEMM_FP8_E5M2;
#define BSGA_GO(G)                                                                                      \
  if (bf16) return e5 ? act_of<G, true, BSGEMM_FP8_E5M2, BWD>(act, p, st, dev)                              \
                      : act_of<G, true, BSGEMM_FP8_E4M3, BWD>(act, p, st, dev);                             \
  return e5 ? act_of<G, false, BSGEMM_FP8_E5M2, BWD>(act, p, st, dev) : act_of<G, false, BSGEMM_FP8_E4M3, BWD>(act, p, st, dev)
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
  return bsga::run<false>(src_dtype, fp8_format, activation, gran, p, static_cast<cudaStream_t>(stream), dev);
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
  st = bsga::run<true>(src_dtype, fp8_format, activation, gran, p, s, dev);
  if (st != BSGEMM_OK || need == 0) return st;
  return bsgr::launch_column_sum(p.part, static_cast<int>(bsga::parts_of(rows, gran)), cols, dbias, s);
}

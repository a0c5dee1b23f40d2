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
// Both run in the block kernel of bsgemm_blocks.cuh. B200, 8192 x 14336 BF16,
// g = 128: GELU 74.7 us (0.72 of the copy rate), its gradient with dbias 117 us
// (0.76), both held by instruction issue; ReLU is at the memory's rate (8192 x
// 8192: 31.6 us, 0.97). Of the first two 7 us each are the quotients' correction
// (bsgemm_rows.cuh), which gives the codes of the correctly rounded quotients.
#include "bsgemm_blocks.cuh"
#include "bsgemm_gelu.cuh"

namespace bsga {

using namespace bsgr;
using namespace bsgg;

enum { kNone = BSGEMM_ACT_NONE, kRelu = BSGEMM_ACT_RELU, kGelu = BSGEMM_ACT_GELU };

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

template <int ACT>
struct Forward {
  static constexpr int kInputs = 1;
  static constexpr bool kSums = false;
  template <int NP>
  struct Rows {};
  struct Cols {};
  template <int NP>
  __device__ __forceinline__ Rows<NP> rows(int64_t, int, int) const {
    return {};
  }
  __device__ __forceinline__ Cols cols(int, bool) const { return {}; }
  template <int NP>
  __device__ __forceinline__ void apply(const Rows<NP>&, const Cols&, int, float2 (&v)[4], const float2 (&)[4]) const {
    act_run<ACT>(v);
  }
};

template <int ACT>
struct Backward {
  static constexpr int kInputs = ACT == kNone ? 1 : 2;
  static constexpr bool kSums = true;
  template <int NP>
  struct Rows {};
  struct Cols {};
  template <int NP>
  __device__ __forceinline__ Rows<NP> rows(int64_t, int, int) const {
    return {};
  }
  __device__ __forceinline__ Cols cols(int, bool) const { return {}; }
  template <int NP>
  __device__ __forceinline__ void apply(const Rows<NP>&, const Cols&, int, float2 (&v)[4], const float2 (&z)[4]) const {
    if constexpr (ACT != kNone) slope_run<ACT>(v, z);
  }
};

// Rows of partial column sums of a backward call.
inline int64_t parts_of(int64_t rows, int gran) { return (rows + gran - 1) / gran * (gran == 256 ? 4 : 1); }

template <template <int> typename Op>
bsgemm_status run(int src, int fmt, int act, int gran, BlockParams& p, cudaStream_t st, const bsg_host::DeviceInfo& dev) {
  const bool bf16 = src == BSGEMM_SRC_BF16;
#define BSGA_GO(ACT) \
  return bf16 ? launch_blocks<true>(gran, fmt, p, Op<ACT>{}, st, dev) : launch_blocks<false>(gran, fmt, p, Op<ACT>{}, st, dev)
  if (act == kGelu) BSGA_GO(kGelu);
  if (act == kRelu) BSGA_GO(kRelu);
  // forward without an activation is the quantiser's own call
  if constexpr (Op<kNone>::kSums) BSGA_GO(kNone);
#undef BSGA_GO
  return BSGEMM_ERR_INVALID_ARG;
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
  bsgr::BlockParams p{};
  p.in0 = z;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.rows = rows;
  p.cols = cols;
  return bsga::run<bsga::Forward>(src_dtype, fp8_format, activation, gran, p, static_cast<cudaStream_t>(stream), dev);
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
  bsgr::BlockParams p{};
  p.in0 = dout;
  p.in1 = z;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.part = need > 0 ? static_cast<float*>(workspace) : dbias;   // one row of sums is the result itself
  p.rows = rows;
  p.cols = cols;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = bsga::run<bsga::Backward>(src_dtype, fp8_format, activation, gran, p, s, dev);
  if (st != BSGEMM_OK || need == 0) return st;
  return bsgr::launch_column_sum(p.part, static_cast<int>(bsga::parts_of(rows, gran)), cols, dbias, s, dev);
}

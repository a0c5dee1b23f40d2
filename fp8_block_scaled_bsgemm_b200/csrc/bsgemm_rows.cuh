// Pieces shared by the row-wise kernels around the GEMM (bsgemm_norm.cu,
// bsgemm_act.cu): runs of 8 consecutive columns, packed FP32 arithmetic and
// the FP8 encoding.
//
// All of these kernels move far more bytes than they compute, so a thread's
// unit of work is a run: 16 bytes of BF16 or 32 bytes of FP32, loaded and
// stored as 16-byte words; 8 codes are stored as one 8-byte word. Rows are
// multiples of 16 columns, so a run lies wholly inside the matrix or outside.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bsgemm.h"
#include "bsgemm_host.h"
#include "ptx.cuh"

namespace bsgr {

constexpr int kVec = 8;  // columns per run

// A run as it lies in memory; widened to FP32 on use (a BF16 run held this
// way costs 4 registers rather than 8).
template <bool BF16>
struct Run {
  uint4 w[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Run<BF16> zero_run() {
  Run<BF16> r;
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = make_uint4(0, 0, 0, 0);
  return r;
}

// BF16 runs are loaded through L2 only: each is read once per pass. An FP32 run
// takes two loads, each of which touches half of every 32-byte sector, so the
// second finds its half in L1.
template <bool BF16>
__device__ __forceinline__ Run<BF16> load_run(const void* base, int64_t elem) {
  Run<BF16> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + elem * (BF16 ? 2 : 4));
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = BF16 ? __ldcg(p + h) : __ldca(p + h);
  return r;
}

// The same for data that is not read again soon: first to leave L2.
template <bool BF16>
__device__ __forceinline__ Run<BF16> load_run_once(const void* base, int64_t elem) {
  Run<BF16> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + elem * (BF16 ? 2 : 4));
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = __ldcs(p + h);
  return r;
}

template <bool BF16>
__device__ __forceinline__ void store_run(void* base, int64_t elem, const Run<BF16>& r) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + elem * (BF16 ? 2 : 4));
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) p[h] = r.w[h];
}

// The run's columns as four FP32 pairs (exact).
template <bool BF16>
__device__ __forceinline__ void widen(const Run<BF16>& r, float2 (&v)[4]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[2 * h] = make_float2(__uint_as_float(r.w[h].x), __uint_as_float(r.w[h].y));
      v[2 * h + 1] = make_float2(__uint_as_float(r.w[h].z), __uint_as_float(r.w[h].w));
    }
  }
}

// Four FP32 pairs as a run of the type: one rounding to nearest even for BF16.
template <bool BF16>
__device__ __forceinline__ Run<BF16> narrow(const float2 (&v)[4]) {
  Run<BF16> r;
  if constexpr (BF16) {
    r.w[0] = make_uint4(bsg::pack_bf16x2(v[0].x, v[0].y), bsg::pack_bf16x2(v[1].x, v[1].y),
                        bsg::pack_bf16x2(v[2].x, v[2].y), bsg::pack_bf16x2(v[3].x, v[3].y));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      r.w[h] = make_uint4(__float_as_uint(v[2 * h].x), __float_as_uint(v[2 * h].y),
                          __float_as_uint(v[2 * h + 1].x), __float_as_uint(v[2 * h + 1].y));
  }
  return r;
}

// Pairwise FP32 arithmetic, one instruction per pair, each element rounded once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <int FMT>
constexpr float kFmax = FMT == BSGEMM_FP8_E5M2 ? 57344.0f : 448.0f;

// A block's scale and its reciprocal, each thread for itself.
//   s = RN(amax / FMAX), or 1 where that is 0 (an empty block, or one whose
//       amax / FMAX is below the smallest FP32 value);
//   rcp = RN(1 / s), or 0 where amax lies outside the range that makes both
//       quotients safe (the codes then take divisions).
// The quotient by the constant is the product with its rounded reciprocal and
// one correction by the exact remainder (Markstein): correctly rounded where
// neither the quotient nor the remainder is near FP32's smallest values, which
// the threshold keeps away; below it the division itself. The threshold keeps
// quotients()'s remainders exact too: a quotient that is not below every border
// between codes is at least 2^-17 (E5M2; E4M3 2^-10), so its value is at least
// 2^-17 * 2^-64 / 57344 > 2^-97, whose remainder is a multiple of 2^-145.
constexpr float kSmallAmax = 0x1p-64f;

struct Scale {
  float s, rcp;
};

template <int FMT>
__device__ __forceinline__ Scale block_scale(float amax) {
  constexpr float inv = 1.0f / kFmax<FMT>;
  Scale r;
  if (amax >= kSmallAmax && amax < 0x1p127f) {
    const float q = amax * inv;
    r.s = __fmaf_rn(__fmaf_rn(-q, kFmax<FMT>, amax), inv, q);
    r.rcp = __frcp_rn(r.s);
  } else {
    const float q = __fdiv_rn(amax, kFmax<FMT>);
    r.s = q > 0.f ? q : 1.f;
    r.rcp = q > 0.f ? 0.f : 1.f;
  }
  return r;
}

// v / s of a run, negated, where s.rcp > 0: the product with the reciprocal and
// Markstein's correction by its remainder, whose FP8 codes are those of the
// correctly rounded quotients (tests/block_quotient_model.c: every scale beside
// every border between codes). With the product alone a value beside a border
// could take the code on the border's other side. The signs are turned so that a
// zero keeps its own without a negation per value; the code's bit is turned back.
__device__ __forceinline__ void quotients(float2 (&v)[4], const Scale& s) {
  const float2 nr = both(-s.rcp);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = mul2(v[i], nr);
    v[i] = bsg::ffma2(bsg::ffma2(p, both(s.s), v[i]), nr, p);
  }
}

// FP8 codes of four values, the first in the lowest byte: round to nearest even,
// saturating. (As one assembly block the two conversions write the halves of the
// word themselves; through the 16-bit intrinsic each pair took further masks.)
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float2 a, float2 b) {
  uint32_t r;
  if constexpr (FMT == BSGEMM_FP8_E5M2)
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Stores the codes of v / s where s.rcp > 0 (WHOLE: the caller knows), else by
// divisions.
template <int FMT, bool WHOLE = false>
__device__ __forceinline__ void store_codes(uint8_t* q, float2 (&v)[4], const Scale& s) {
  uint32_t sign = 0;
  if (WHOLE || s.rcp > 0.f) {
    quotients(v, s);
    sign = 0x80808080u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__fdiv_rn(v[i].x, s.s), __fdiv_rn(v[i].y, s.s));
  }
  *reinterpret_cast<uint2*>(q) = make_uint2(encode4<FMT>(v[0], v[1]) ^ sign, encode4<FMT>(v[2], v[3]) ^ sign);
}

// Largest of a (not negative) and the run's magnitudes, two values to an
// instruction; NaNs are passed over.
__device__ __forceinline__ float max_abs(float a, const float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float b = a;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(b), "f"(v[i].x), "f"(v[i].y));
  }
  return a;
}

// Store a float to a CTA's shared memory in the cluster (a shared::cluster address).
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// ------------------------------------------------------------------ host side

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Sizes, types and device of a row-wise call; nothing is launched on an error.
inline bsgemm_status check_rows(int src_dtype, int64_t rows, int64_t cols) {
  if (src_dtype != BSGEMM_SRC_F32 && src_dtype != BSGEMM_SRC_BF16) return BSGEMM_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || rows > (1 << 30) || cols > (1 << 24)) return BSGEMM_ERR_INVALID_ARG;
  return cols % 16 ? BSGEMM_ERR_MISALIGNED : BSGEMM_OK;
}

// A buffer of a call, for the check of overlaps.
struct Span {
  const void* p;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}
// True where an output shares memory with another output or with an input.
template <int NO, int NI>
bool any_overlap(const Span (&out)[NO], const Span (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = i + 1; j < NO; ++j)
      if (overlap(out[i], out[j])) return true;
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
  }
  return false;
}
// `b`, or no buffer where it is the very buffer `a` (allowed where a call says so).
inline Span unless_same(const Span& a, const Span& b) { return a.p == b.p ? Span{nullptr, 0} : b; }

inline size_t blocks_bytes(int64_t rows, int64_t cols, int g) {
  return static_cast<size_t>((rows + g - 1) / g) * static_cast<size_t>((cols + g - 1) / g) * sizeof(float);
}

// Adds up `parts` rows of partial sums in order: out[c] = sum_i part[i][c].
bsgemm_status launch_column_sum(const float* part, int parts, int64_t cols, float* out, cudaStream_t stream,
                                const bsg_host::DeviceInfo& dev);

// Once per device, before Kern's first launch with `smem` bytes of dynamic
// shared memory (the same in every call of a kernel).
template <auto Kern>
bool prepare_rows(const bsg_host::DeviceInfo& dev, int smem) {
  static bsg_host::PerDeviceOnce setup;
  if (setup.done(dev.ordinal)) return true;
  if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      // clusters of 16 are beyond the portable size
      cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return false;
  setup.mark(dev.ordinal);
  return true;
}

struct RowsLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  RowsLaunch(int64_t grid, int threads, int smem, int cluster, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // the kernel's set-up may overlap the end of the stream's previous kernel
    // (every kernel here waits for it before touching global memory)
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = cluster > 1 ? attr : attr + 1;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
};

template <auto Kern, typename... A>
bsgemm_status launch_rows(const bsg_host::DeviceInfo& dev, int64_t grid, int threads, int smem, int cluster,
                          cudaStream_t stream, A... args) {
  if (grid < 1 || grid > 0x7FFFFFFFll) return BSGEMM_ERR_INVALID_ARG;
  if (!prepare_rows<Kern>(dev, smem)) return BSGEMM_ERR_CUDA;
  RowsLaunch l(grid, threads, smem, cluster, stream);
  const cudaLaunchConfig_t& cfg = l.cfg;
  if (cudaLaunchKernelEx(&cfg, Kern, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return BSGEMM_ERR_CUDA;
  }
  return BSGEMM_OK;
}

}  // namespace bsgr

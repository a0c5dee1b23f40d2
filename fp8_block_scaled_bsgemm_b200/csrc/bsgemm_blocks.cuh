// The kernel that turns a matrix into FP8 codes and block scales while it
// computes each value: activations and their gradients (bsgemm_act.cu) and the
// second half of the norm (bsgemm_norm.cu). What a value is comes from Op:
//   Op::kInputs      matrices read (1 or 2)
//   Op::kSums        whether the values' column sums are wanted (Params.part)
//   Op::Rows<NP>     what the thread's NP rows of a block need, from op.rows<NP>(
//                    first row, rows that exist, distance between rows)
//   Op::Cols         what its column needs, from op.cols(column, whether it exists)
//   op.apply(rows, cols, j, v, z)   v: the run of the thread's j-th row from the
//                    first input, replaced by its values; z: the second input's.
//                    Outside the matrix both are 0 and so must the value be.
//
// Per g x g block: s = amax / FMAX (1 if that is 0), q = FP8 code of value / s.
// One CTA takes a block with g <= 128; a cluster of four one with g = 256, 64 of
// its rows each. A thread computes its values once, keeps them in registers
// past the block's amax, and encodes them.
#pragma once
#include <atomic>

#include "bsgemm_host.h"
#include "bsgemm_rows.cuh"

namespace bsgr {

template <int G>
constexpr int kParts = G == 256 ? 4 : 1;   // CTAs to a block
template <int G>
constexpr int kThreads = G == 64 ? 256 : 512;
template <int G>
constexpr int kCtasPerSm = G == 64 ? 4 : 2;

// A thread's runs of a block pass through shared memory (cp.async into places
// that its warp alone reads, so no barrier of the CTA is needed), which keeps
// the next block's loads in flight while this one is computed without holding
// them in registers. Two buffers where they fit beside a second CTA, else one, refilled
// once the block's values are in registers; none for the widest case.
template <int G, bool BF16, bool IN2>
constexpr int kBufBytes = kThreads<G> * (G / kParts<G> / (kThreads<G> / (G / kVec))) * (BF16 ? 16 : 32) * (IN2 ? 2 : 1);
template <int G, bool BF16, bool IN2>
constexpr int kBufs = kBufBytes<G, BF16, IN2> * kCtasPerSm<G> * 2 <= 192 * 1024 ? 2
                      : kBufBytes<G, BF16, IN2> * kCtasPerSm<G> <= 192 * 1024 ? 1 : 0;

struct BlockParams {
  const void* in0;
  const void* in1;     // where Op reads two
  uint8_t* q;
  float* scales;
  float* part;         // column sums of each CTA's rows [row blocks x CTAs to a block][cols], or null
  int64_t rows, cols;
  int row_blocks, col_blocks;
  int step_rb, step_cb;   // from a CTA's block to its next: rows and columns of blocks
  int backwards;          // rows of blocks are taken from the last to the first
};

// A walk over the matrix's blocks in row-major order, without divisions. rb
// counts rows of blocks from the first taken; row() is the one meant.
struct Walk {
  int rb, cb;
  __device__ __forceinline__ int row(const BlockParams& p) const {
    return p.backwards ? p.row_blocks - 1 - rb : rb;
  }
  __device__ __forceinline__ void next(const BlockParams& p) {
    rb += p.step_rb;
    cb += p.step_cb;
    if (cb >= p.col_blocks) {
      cb -= p.col_blocks;
      ++rb;
    }
  }
};

// Copies 16 bytes into shared memory, zeros (and no access) where they lie
// outside the matrix (WHOLE: they do not).
template <bool WHOLE>
__device__ __forceinline__ void fetch16(uint32_t dst, const char* src, bool in) {
  if constexpr (WHOLE)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// One run for each of L neighbouring threads, in shared memory as in global
// memory: 16 or 32 bytes a thread from `dst` on. A BF16 run is 16 bytes and its
// thread copies it. An FP32 run is two halves; if its thread copied both, each
// copy of a warp would touch half of every 32-byte sector and fetch it twice. So
// the group's 2 L halves are copied in address order, thread i taking halves i
// and i + L (L * 16 bytes on). `src` is the thread's first 16 bytes, `in` and
// `in2` whether its pieces exist.
template <bool BF16, bool WHOLE, int T, int L>
__device__ __forceinline__ void fetch_run(uint32_t dst, int tid, const char* src, bool in, bool in2) {
  if constexpr (BF16) {
    fetch16<WHOLE>(dst + tid * 16, src, in);
  } else {
    static_assert(L >= 8 && L <= 32, "a group lies within a warp");
    dst += (tid - tid % L) * 32 + tid % L * 16;
    fetch16<WHOLE>(dst, src, in);
    fetch16<WHOLE>(dst + L * 16, src + (in2 || WHOLE ? L * 16 : 0), in2);
  }
}
// The thread's run, past fetch_wait (and a __syncwarp for FP32). Of an FP32 run
// every other group of four threads reads the second half first, so that the
// eight threads of a bank cycle, 32 bytes apart, meet in no bank.
template <bool BF16, int T>
__device__ __forceinline__ Run<BF16> fetched_run(const uint4* at, int tid) {
  Run<BF16> r;
  if constexpr (BF16) {
    r.w[0] = at[tid];
  } else {
    const int flip = (tid >> 2) & 1;
    const uint4 x = at[2 * tid + flip], y = at[2 * tid + (flip ^ 1)];
    r.w[0] = flip ? y : x;
    r.w[1] = flip ? x : y;
  }
  return r;
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Persistent: CTA (or cluster) k takes blocks k, k + grid, ... in row-major
// order.
template <int G, bool BF16, int FMT, typename Op>
__global__ void __launch_bounds__(kThreads<G>, kCtasPerSm<G>)
    block_quant_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ Op op) {
  constexpr int T = kThreads<G>;
  constexpr int P = kParts<G>;
  constexpr int L = G / kVec;          // threads to a row
  constexpr int RP = T / L;            // rows at a time
  constexpr int NP = G / P / RP;       // rows a thread holds
  constexpr int W = T / 32;
  constexpr bool IN2 = Op::kInputs == 2;
  constexpr bool SUMS = Op::kSums;
  constexpr int kBuf = kBufs<G, BF16, IN2>;
  constexpr int kRun = BF16 ? 16 : 32;
  static_assert(NP * RP * P == G, "the rows of a block are dealt out evenly");
  extern __shared__ uint4 fetched[];   // [kBuf][inputs][NP][T] runs
  __shared__ float warp_max[2][W];
  __shared__ float part_max[2][P];
  // column sums of each group of L threads; a run's first four columns lie in
  // the first half of a row, its others in the second (no bank conflicts)
  __shared__ float4 col_sum[SUMS ? 2 : 1][SUMS ? RP : 1][2][SUMS ? L : 1];

  constexpr int kElem = BF16 ? 2 : 4;
  const int tid = threadIdx.x;
  const int part = static_cast<int>(blockIdx.x % P);   // the CTA's rank in its cluster
  const int row0 = part * (G / P) + tid / L;           // the thread's first row of a block
  const int col8 = (tid % L) * kVec;
  const int cols = static_cast<int>(p.cols);           // at most 2^24, rows at most 2^30
  const int rows = static_cast<int>(p.rows);
  // the thread's elements within a row of blocks: a block's first element is the
  // same for all threads, and 256 rows of 2^24 columns are counted in 32 bits
  uint32_t off[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) off[j] = static_cast<uint32_t>(row0 + j * RP) * cols + col8;
  // the first column that the thread copies: its own run's for BF16, see fetch_run
  const int copy_col = BF16 ? col8 : col8 / 2;
  auto first_of = [&](const Walk& w) { return static_cast<int64_t>(w.row(p)) * G * p.cols + w.cb * G; };
  // row j * RP of the thread exists in block w if below this
  auto left_of = [&](const Walk& w) { return w.cb * G + col8 < cols ? rows - w.row(p) * G - row0 : 0; };
  // the whole block lies inside the matrix
  auto whole_of = [&](const Walk& w) { return (w.cb + 1) * G <= cols && rows - w.row(p) * G >= G; };

  if constexpr (P > 1) bsg::cluster_open_arrive();
  bsg::grid_launch_dependents();
  bsg::grid_dependency_wait();

  const uint32_t runs = kBuf > 0 ? bsg::smem_addr(fetched) : 0;
  auto slot = [&](int buf, int input, int j) -> uint32_t {
    return runs + ((buf * (IN2 ? 2 : 1) + input) * NP + j) * (T * kRun);
  };
  const char* in0 = static_cast<const char*>(p.in0);
  const char* in1 = static_cast<const char*>(p.in1);
  auto fetch = [&](const Walk& w, int buf) {
    if (w.rb < p.row_blocks) {
      const int64_t first = first_of(w) - (col8 - copy_col);
      const char* src0 = in0 + first * kElem;
      const char* src1 = in1 + (IN2 ? first * kElem : 0);
      if (whole_of(w)) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const uint64_t e = static_cast<uint64_t>(off[j]) * kElem;
          fetch_run<BF16, true, T, L>(slot(buf, 0, j), tid, src0 + e, true, true);
          if constexpr (IN2) fetch_run<BF16, true, T, L>(slot(buf, 1, j), tid, src1 + e, true, true);
        }
      } else {
        const int c = w.cb * G + copy_col, left = rows - w.row(p) * G - row0;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const bool in = j * RP < left && c < cols, in2 = j * RP < left && c + L * 4 < cols;
          const uint64_t e = static_cast<uint64_t>(off[j]) * kElem;
          fetch_run<BF16, false, T, L>(slot(buf, 0, j), tid, in ? src0 + e : in0, in, in2);
          if constexpr (IN2) fetch_run<BF16, false, T, L>(slot(buf, 1, j), tid, in ? src1 + e : in1, in, in2);
        }
      }
    }
    fetch_commit();
  };
  auto fetched_of = [&](int buf, int input, int j) {
    return fetched_run<BF16, T>(fetched + ((buf * (IN2 ? 2 : 1) + input) * NP + j) * (T * kRun / 16), tid);
  };

  Walk w{static_cast<int>(blockIdx.x / P) / p.col_blocks, static_cast<int>(blockIdx.x / P) % p.col_blocks};
  auto rows_of = [&](const Walk& at) {
    return op.template rows<NP>(static_cast<int64_t>(at.row(p)) * G + row0, rows - at.row(p) * G - row0, RP);
  };
  if constexpr (kBuf > 0) fetch(w, 0);
  if constexpr (P > 1) bsg::cluster_open_wait();
  int par = 0;   // parity of the block: which copy of the exchanged values it uses
  for (; w.rb < p.row_blocks; par ^= 1) {
    const int64_t first = first_of(w);
    const int left = left_of(w);
    const bool whole = whole_of(w);
    const int64_t blk = static_cast<int64_t>(w.row(p)) * p.col_blocks + w.cb;
    const int c0 = w.cb * G;
    const int64_t part_row = static_cast<int64_t>(w.row(p)) * P + part;
    const typename Op::template Rows<NP> of_rows = rows_of(w);
    const typename Op::Cols of_cols = op.cols(c0 + col8, left > 0);
    w.next(p);
    const int buf = kBuf == 2 ? par : 0;
    if constexpr (kBuf == 2) {
      fetch(w, par ^ 1);
      fetch_wait<1>();
    } else if constexpr (kBuf == 1) {
      fetch_wait<0>();
    }
    if constexpr (!BF16 && kBuf > 0) __syncwarp();   // the warp's other threads' copies
    float2 v[NP][4];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      Run<BF16> a, b;
      if constexpr (kBuf > 0) {
        a = fetched_of(buf, 0, j);
        if constexpr (IN2) b = fetched_of(buf, 1, j);
      } else {
        a = b = zero_run<BF16>();
        if (j * RP < left) {
          a = load_run<BF16>(in0, first + off[j]);
          if constexpr (IN2) b = load_run<BF16>(in1, first + off[j]);
        }
      }
      float2 z[4];
      widen<BF16>(a, v[j]);
      if constexpr (IN2) widen<BF16>(b, z);
      op.apply(of_rows, of_cols, j, v[j], z);
      amax = max_abs(amax, v[j]);
    }
    // magnitudes are not negative, so their bit patterns order as they do
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if ((tid & 31) == 0) warp_max[par][tid / 32] = amax;
    if constexpr (SUMS) {
      if (p.part != nullptr) {
        float2 s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i] = v[0][i];
#pragma unroll
          for (int j = 1; j < NP; ++j) s[i] = add2(s[i], v[j][i]);
        }
        col_sum[par][tid / L][0][tid % L] = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
        col_sum[par][tid / L][1][tid % L] = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
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
    uint8_t* q = p.q + first;
    if (whole && s.rcp > 0.f) {
#pragma unroll
      for (int j = 0; j < NP; ++j) store_codes<FMT, true>(q + off[j], v[j], s);
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (j * RP < left) store_codes<FMT>(q + off[j], v[j], s);
    }
    if constexpr (SUMS) {
      if (p.part != nullptr && tid < G && c0 + tid < cols) {
        const float* of = reinterpret_cast<const float*>(&col_sum[par][0][(tid >> 2) & 1][tid >> 3]) + (tid & 3);
        float sum = of[0];
#pragma unroll
        for (int k = 1; k < RP; ++k) sum += of[k * G];
        p.part[part_row * p.cols + c0 + tid] = sum;
      }
    }
  }
  // no copy is in flight here: fetches past the last block are empty, and the
  // last block's were waited for
}

// Launches the kernel on p's matrices (p's sizes in blocks are filled in here).
template <int G, bool BF16, int FMT, typename Op>
bsgemm_status launch_blocks(BlockParams& p, const Op& op, cudaStream_t stream, const bsg_host::DeviceInfo& dev) {
  constexpr bool IN2 = Op::kInputs == 2;
  constexpr int kSmem = kBufBytes<G, BF16, IN2> * kBufs<G, BF16, IN2>;
  p.row_blocks = static_cast<int>((p.rows + G - 1) / G);
  p.col_blocks = static_cast<int>((p.cols + G - 1) / G);
  // Blocks taken at the same time: no more clusters than can be resident, since
  // the rest would begin when the others have ended (a GPC's SMs do not hold a
  // whole number of clusters: 74 of them for 148 SMs doubled the time).
  int64_t units = int64_t{dev.num_sms} * kCtasPerSm<G>;
  if constexpr (kParts<G> > 1) {
    static std::atomic<int> resident[64];
    const int slot = dev.ordinal >= 0 && dev.ordinal < 64 ? dev.ordinal : -1;
    int n = slot >= 0 ? resident[slot].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
      constexpr auto kern = block_quant_kernel<G, BF16, FMT, Op>;
      if (!prepare_rows<block_quant_kernel<G, BF16, FMT, Op>>(dev, kSmem)) return BSGEMM_ERR_CUDA;
      RowsLaunch l(units, kThreads<G>, kSmem, kParts<G>, stream);
      l.cfg.numAttrs = 1;   // the cluster shape alone decides residency
      if (cudaOccupancyMaxActiveClusters(&n, kern, &l.cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return BSGEMM_ERR_CUDA;
      }
      if (slot >= 0) resident[slot].store(n, std::memory_order_relaxed);
    }
    units = n;
  }
  const int64_t blocks = static_cast<int64_t>(p.row_blocks) * p.col_blocks;
  if (units > blocks) units = blocks;
  p.step_rb = static_cast<int>(units / p.col_blocks);
  p.step_cb = static_cast<int>(units % p.col_blocks);
  return launch_rows<block_quant_kernel<G, BF16, FMT, Op>>(dev, units * kParts<G>, kThreads<G>, kSmem, kParts<G>,
                                                           stream, p, op);
}

// The same for run-time sizes and formats.
template <bool BF16, typename Op>
bsgemm_status launch_blocks(int gran, int fmt, BlockParams& p, const Op& op, cudaStream_t stream,
                            const bsg_host::DeviceInfo& dev) {
#define BSGR_GO(G)                                                                                   \
  return fmt == BSGEMM_FP8_E5M2 ? launch_blocks<G, BF16, BSGEMM_FP8_E5M2, Op>(p, op, stream, dev)   \
                                : launch_blocks<G, BF16, BSGEMM_FP8_E4M3, Op>(p, op, stream, dev)
  switch (gran) {
    case 64:  BSGR_GO(64);
    case 128: BSGR_GO(128);
    default:  BSGR_GO(256);
  }
#undef BSGR_GO
}

}  // namespace bsgr

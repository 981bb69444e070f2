// nm_grad.cu -- gradients of the gated feed-forward block (nm_gated_backward).
//
//   dp = (dY u act'(g), dY act(g))      elementwise, [T][2 n_ff]
//   dX = dp Wm                          T x k, summed over 2 n_ff
//   dW = dp^T X                         2 n_ff x k, summed over T
//   dbias = sum over T of dp
//
// The pattern of Wm runs along k, the axis dX keeps and dW produces, so neither
// product is one the 2:4 tensor core could take: both are dense 16-bit products
// of operands that lie in memory the wrong way round for a K-major operand (dp
// and X are summed along their rows for dW, Wm along its rows for dX).  The tensor
// core reads MN-major operands as well, so nothing is transposed: tensor copies
// bring 64-wide runs of the kept axis, 64 summed rows each.
#include <algorithm>
#include <cstdlib>

#include "nm_act.cuh"
#include "nm_api_internal.h"
#include "nm_device.cuh"
#include "nm_launch.cuh"
#include "nm_stage.cuh"
#include "nm_unpack.cuh"

namespace nm {
namespace {

// ------------------------------------------------------------------ dp and dbias

constexpr int kDpCols = 256;  // columns of each half per block
constexpr int kDpWarps = 8;

template <int DT>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (DT == DT_BF16) return __uint_as_float((uint32_t)v << 16);
  return __half2float(__ushort_as_half(v));
}
template <int DT>
__device__ __forceinline__ uint16_t to_16(float v) {
  if constexpr (DT == DT_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

// (Loads here are coherent ones: P may come from the kernel just before, beside
// which this one may have started.)
// Eight of this lane's columns of one row: consecutive (VEC: 16-byte accesses) or
// 32 apart (any alignment).
template <bool VEC>
__device__ __forceinline__ int dp_col(int lane, int j) {
  return VEC ? lane * 8 + j : j * 32 + lane;
}
template <int DT, bool VEC>
__device__ __forceinline__ void dp_load(const uint16_t* row, int f0, int F, int lane, float (&v)[8]) {
  if constexpr (VEC) {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (f0 + lane * 8 < F) q = __ldcs(reinterpret_cast<const uint4*>(row + f0 + lane * 8));  // read once: leave L2 to dp
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = to_f32<DT>((uint16_t)(w[i] & 0xFFFFu));
      v[2 * i + 1] = to_f32<DT>((uint16_t)(w[i] >> 16));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int f = f0 + dp_col<false>(lane, j);
      v[j] = f < F ? to_f32<DT>(__ldca(row + f)) : 0.0f;
    }
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ void dp_store(uint16_t* row, int f0, int F, int lane, const float (&v)[8]) {
  if constexpr (VEC) {
    constexpr int OT = DT == DT_F16 ? OUT_F16 : OUT_BF16;
    if (f0 + lane * 8 < F)
      *reinterpret_cast<uint4*>(row + f0 + lane * 8) = make_uint4(
          pack_pair<OT>(v[0], v[1]), pack_pair<OT>(v[2], v[3]), pack_pair<OT>(v[4], v[5]), pack_pair<OT>(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int f = f0 + dp_col<false>(lane, j);
      if (f < F) row[f] = to_16<DT>(v[j]);
    }
  }
}

// The masked dense weight, unpacked by the first blocks of the same launch (dX
// reads it with dp): Wm null or blocks = 0 when dX is not asked for.
struct UnpackArgs {
  const uint8_t* bpack;
  uint16_t* Wm;
  long long units, K;
  int img, n_kb, n_ff, blocks;
};

// dp of row t, this lane's eight columns from f0: g the gate half, u the up half.
template <int DT, bool VEC>
__device__ __forceinline__ void dp_row(const uint16_t* __restrict__ P, const uint16_t* __restrict__ dY, int t, int f0, int F,
                                       int lane, int act, float (&g)[8], float (&u)[8]) {
  const uint16_t* prow = P + (size_t)t * 2 * F;
  float dy[8];
  dp_load<DT, VEC>(prow, f0, F, lane, g);
  dp_load<DT, VEC>(prow + F, f0, F, lane, u);
  dp_load<DT, VEC>(dY + (size_t)t * F, f0, F, lane, dy);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a, d;
    act_slope(g[j], act, a, d);
    g[j] = __fmul_rn(__fmul_rn(dy[j], u[j]), d);
    u[j] = __fmul_rn(dy[j], a);
  }
}

// Range of dp in fp16.  dY and u are fp16 values, their product is not: above 65504 it
// would become infinite (and with a zero of the pruned weight NaN), below 2^-24 zero,
// where fp32 keeps it and the sums it goes into may well be representable.  So each block
// leaves its largest finite |dp|, and where the largest of all is outside [2^-4, 2^15)
// gated_dp_scale_kernel writes dp again, times the power of two that brings it to [2^14,
// 2^15); the products divide by it before they round.  An element is off by its rounding
// and 2^-21 of the largest |dp| at most.  The whole call in graphs, before, in range and
// outside it: 1379 x 768 -> 2 x 2051 30.3, 34.0, 39.7 us; 6304 x 1024 -> 2 x 4096 208,
// 210, 262.  (A pass that only looks for the maximum first would cost the last figures
// always; one block an SM here instead of four the same in range, 322 outside.)
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}
// The power of two, as its exponent, that dp is stored times (0 without any finite non-zero).
__device__ __forceinline__ int dp_exponent(uint32_t peak) {
  const int e = (int)(peak >> 23) - 127;
  return peak == 0u || (e >= -4 && e <= 14) ? 0 : min(14 - e, 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// One pass over P and dY: dp [T][2][pitch] in the handle's type (columns n_ff .. pitch
// are never read; the rounding is that of the products' tensor-core operand, as in
// mixed-precision training: it adds as much error, by rms, as the rounding of dX and dW
// themselves, and two terms of dp would double the products) and, with `part`, the fp32
// column sums of this block's rows ([row block][2][n_ff]), each warp's rows in
// ascending order, the warps in order.  Memory bound: 48-51 us for 6304 x 2 x 4096
// bf16 with the weight unpacked beside it (246 MB of DRAM traffic, 5 TB/s).
// BIAS is its own instance: the sums' registers cost the plain one a third of its
// warps.  With `peak` (fp16): this block's largest finite |dp|, as bits.
template <int DT, bool VEC, bool BIAS>
__global__ void __launch_bounds__(32 * kDpWarps, BIAS ? 3 : 4)
    gated_dp_kernel(const uint16_t* __restrict__ P, const uint16_t* __restrict__ dY, int T, int F, int pitch, int act,
                    uint16_t* __restrict__ dp, float* __restrict__ part, uint32_t* __restrict__ peak, int block_rows,
                    int col_blocks, const UnpackArgs un) {
  __shared__ float sums[BIAS ? kDpWarps : 1][2][kDpCols];
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x < un.blocks) {
    const long long unit = (long long)blockIdx.x * (32 * kDpWarps) + threadIdx.x, per_row = (un.K + 15) / 16;
    if (unit < un.units) {
      const long long r = unit / per_row;
      unpack_unit<DT>(un.bpack, un.n_ff, un.K, un.img, un.n_kb, un.Wm, r, (unit - r * per_row) * 16);
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = (int)blockIdx.x - un.blocks, row_block = block / col_blocks;
  const int f0 = (block - row_block * col_blocks) * kDpCols, t0 = row_block * block_rows;
  const int t1 = min(T, t0 + block_rows);
  float sg[8] = {}, su[8] = {};
  [[maybe_unused]] uint32_t top = 0;
  for (int t = t0 + warp; t < t1; t += kDpWarps) {
    float g[8], u[8];
    dp_row<DT, VEC>(P, dY, t, f0, F, lane, act, g, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (BIAS) {
        sg[j] += g[j];
        su[j] += u[j];
      }
      if constexpr (DT == DT_F16) top = max(top, max(finite_bits(g[j]), finite_bits(u[j])));
    }
    uint16_t* out = dp + (size_t)t * 2 * pitch;
    dp_store<DT, VEC>(out, f0, F, lane, g);
    dp_store<DT, VEC>(out + pitch, f0, F, lane, u);
  }
  if constexpr (DT == DT_F16) {
    if (peak) {
      __shared__ uint32_t tops[kDpWarps];
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) tops[warp] = top;
      __syncthreads();
      if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kDpWarps; ++w) top = max(top, tops[w]);
        peak[block] = top;
      }
    }
  }
  if constexpr (BIAS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[warp][0][dp_col<VEC>(lane, j)] = sg[j];
      sums[warp][1][dp_col<VEC>(lane, j)] = su[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kDpCols; i += 32 * kDpWarps) {
      const int z = i / kDpCols, c = i % kDpCols;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kDpWarps; ++w) s += sums[w][z][c];
      if (f0 + c < F) part[((size_t)row_block * 2 + z) * F + f0 + c] = s;
    }
  }
}

// fp16: decides from the blocks' largest |dp| whether dp has to be scaled, leaves the
// factor that undoes it for the products, and if so writes dp again.
template <bool VEC>
__global__ void __launch_bounds__(32 * kDpWarps, 4)
    gated_dp_scale_kernel(const uint16_t* __restrict__ P, const uint16_t* __restrict__ dY, int T, int F, int pitch, int act,
                          uint16_t* __restrict__ dp, const uint32_t* peak, int blocks, int block_rows, int col_blocks,
                          float* __restrict__ undo) {
  __shared__ uint32_t tops[kDpWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t top = 0;
  for (int b = threadIdx.x; b < blocks; b += 32 * kDpWarps) top = max(top, __ldcg(peak + b));
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kDpWarps; ++w) top = max(top, tops[w]);
  const int e = dp_exponent(top);
  if (blockIdx.x == 0 && threadIdx.x == 0) *undo = pow2(-e);
  if (e == 0) return;
  const float scale = pow2(e);
  for (int block = (int)blockIdx.x; block < blocks; block += (int)gridDim.x) {
    const int row_block = block / col_blocks, f0 = (block - row_block * col_blocks) * kDpCols;
    const int t0 = row_block * block_rows, t1 = min(T, t0 + block_rows);
    for (int t = t0 + warp; t < t1; t += kDpWarps) {
      float g[8], u[8];
      dp_row<DT_F16, VEC>(P, dY, t, f0, F, lane, act, g, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] *= scale;
        u[j] *= scale;
      }
      uint16_t* out = dp + (size_t)t * 2 * pitch;
      dp_store<DT_F16, VEC>(out, f0, F, lane, g);
      dp_store<DT_F16, VEC>(out + pitch, f0, F, lane, u);
    }
  }
}

// dbias: a warp adds up the row blocks' sums of four columns, its eight groups of
// four lanes every eighth row block each (eight loads in flight a lane), then the
// groups pairwise: a fixed order whatever the launch.
__device__ __forceinline__ void dbias_columns(const float* __restrict__ part, int n, int row_blocks, int c0, int lane,
                                              float* __restrict__ dbias) {
  const int c = c0 + (lane & 3), group = lane >> 2;
  float run[8] = {};
  if (c < n) {
    for (int b = group; b < row_blocks; b += 64) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (b + 8 * i < row_blocks) run[i] += __ldcg(part + (size_t)(b + 8 * i) * n + c);
    }
  }
  float s = run[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) s += run[i];
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (group == 0 && c < n) dbias[c] = s;
}

// The launch of a call that asks for nothing else; otherwise the products' idle
// epilogue warps do this before their first tile.
__global__ void __launch_bounds__(128) dbias_kernel(const float* __restrict__ part, int n, int row_blocks,
                                                    float* __restrict__ dbias) {
  pdl_launch_dependents();
  pdl_wait();
  dbias_columns(part, n, row_blocks, (int)(blockIdx.x * 4 + (threadIdx.x >> 5)) * 4, threadIdx.x & 31, dbias);
}

// ------------------------------------------------------------------ the two products
//
// One persistent launch computes both: CTA pairs (tcgen05.mma.cta_group::2, M =
// 256, N = BN) walk the tiles of the product with the longer sum first, then
// those of the other (the host splits them evenly over the pairs).
//   dW tile: rows f of one half, columns k; A = dp^T (MN-major), B = X (MN-major)
//   dX tile: rows t,             columns k; A = dp (K-major),     B = Wm (MN-major)
// A stage holds 64 summed elements: 16 KB of A and BN / 2 columns of B per CTA.
// Two accumulators of BN columns; 16-bit output through staged rows.  Every copy
// is zero-filled outside its tensor, so ragged sizes need no masks.
//
// What bounds it: 256-wide tiles run a stage in 0.27 us (512 cycles of MMA) until
// the power cap, 0.33 over seconds; 6304 x 1024 -> 2 x 4096 takes 154 us (1370
// TFLOP/s, 1.48 GHz at 990 W).  Where few pairs work, a 128-wide stage takes
// 0.19-0.2 us, the round trip of a copy over the eight stages in flight.
//
// Long sums.  The tensor core truncates its fp32 accumulator: a step of 16 products
// loses half a unit in the last place on average, so same-sign sums of n products came
// out n / 16 x 2^-24 low (0.17 % at n = 2^18, 0.67 % at 2^20).  An accumulator therefore
// takes kRunKb stages at most, 2^14 products (1.0e-4 low then, a fifth of fp16's half
// unit); the epilogue adds the runs of a longer sum in fp32, rounded to nearest, in
// order: the whole call 255 -> 262 us at 65536 x 768 -> 2 x 512, 1.0 ms as before at 32768
// x 1024 -> 2 x 4096; sums of one run are as they were.
constexpr int kGradKb = 64;
constexpr int kRunKb = 256;
constexpr int kGradEpiWarps = 8;
constexpr int kGradThreads = 64 + 32 * kGradEpiWarps;

template <int BN>
struct GradCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int RUN = kGradKb * 128;            // one 128-byte run of an MN-major operand: 64 rows
  static constexpr int NB = BN / 128;                  // runs of B per CTA
  static constexpr int STAGE = A_BYTES + NB * RUN;
  static constexpr int EPI_BUF = 4096;                 // 32 staged rows of 128 bytes
  static constexpr int EPI_BYTES = kGradEpiWarps * EPI_BUF;
  static constexpr int STAGES_FIT = (227 * 1024 - 1024 - EPI_BYTES) / STAGE;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr int SMEM = STAGES * STAGE + EPI_BYTES + 1024;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int WCOLS = BN / (kGradEpiWarps / 4);
  static_assert(BN == 128 || BN == 256, "tile width");
};

// One of the two products as the kernel sees it.
struct GradSide {
  int tiles, n_nt;   // tiles; column tiles
  int dw;            // 1: dW, 0: dX
  int n_kb;          // stages per tile
  int n_mt;          // row tiles (dW: of one half)
  int splits;        // parts of a tile's sum, of `per_split` stages: units = tiles * splits
  int per_split;
  int slot0;         // splits > 1: where its units' partial tiles start
};

struct GradArgs {
  GradSide side[2];
  int hi;                  // pairs with one more unit of side 0 than the others
  int hi_units, lo_units;  // units of side 1 for those pairs, and for the others
  int F, T, k;
  int kb_half;       // dX: stages per half of 2 n_ff
  // Where few tiles have long sums, a tile is cut into parts on several pairs: they
  // leave fp32 tiles in `partial` ([slot][256][BN]) and grad_join_kernel adds them up.
  float* partial;
  float* runs;             // sums of more than kRunKb stages: each epilogue warp's columns so far
  void *dW, *dX;
  const float* undo;       // fp16: the factor that undoes dp's scaling
  const float* part;       // with dbias: the row blocks' column sums, row_blocks of them
  float* dbias;
  int row_blocks;
  int* err;
  unsigned long long timeout_ns;
};

struct GradUnit {
  int dw, m0, n0, z;
  int kb0, kb1;  // stages of the sum
  int slot;      // part of a split tile: where its fp32 tile goes; else -1
};

// The i-th unit of this pair; false when there is none.  Side 0's units go round
// the pairs; `hi` pairs get one more of them than the others.  Side 1's: first
// lo_units - hi_units rounds over the other pairs alone, then hi_units rounds
// over all (hi_units <= lo_units), the last round cut off at the end of the list.
__host__ __device__ __forceinline__ bool grad_unit(const GradArgs& a, int pair, int pairs, int i, int bn, GradUnit& u) {
  const int n0 = a.side[0].tiles * a.side[0].splits;
  const int q = n0 / pairs + (pair < a.hi ? 1 : 0);
  int s = 0, unit;
  if (i < q) {
    unit = i * pairs + pair;
  } else {
    s = 1;
    int r = i - q;
    const int extra = a.lo_units - a.hi_units, lo_pairs = pairs - a.hi;
    if (pair >= a.hi) {
      if (r < extra) {
        unit = r * lo_pairs + (pair - a.hi);
      } else {
        r -= extra;
        if (r >= a.hi_units) return false;
        unit = extra * lo_pairs + r * pairs + (pair - a.hi);
      }
    } else {
      if (r >= a.hi_units) return false;
      unit = extra * lo_pairs + r * pairs + lo_pairs + pair;
    }
    if (unit >= a.side[1].tiles * a.side[1].splits) return false;
  }
  const GradSide& g = a.side[s];
  const int tile = unit / g.splits, part = unit - tile * g.splits;
  const int nt = tile % g.n_nt, mt = tile / g.n_nt;
  u.dw = g.dw;
  u.kb0 = part * g.per_split;
  u.kb1 = u.kb0 + g.per_split < g.n_kb ? u.kb0 + g.per_split : g.n_kb;
  u.slot = g.splits > 1 ? g.slot0 + unit : -1;
  u.n0 = nt * bn;
  u.z = g.dw ? mt / g.n_mt : 0;
  u.m0 = (g.dw ? mt % g.n_mt : mt) * 256;
  return true;
}

template <int DT, int BN>
__host__ __device__ constexpr uint32_t grad_idesc(bool a_mn) {
  const uint32_t f = DT == DT_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | (1u << 16) | ((uint32_t)(BN >> 3) << 17) |
         ((256u >> 4) << 24);
}

template <int DT, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    grad_pair_kernel(const __grid_constant__ CUtensorMap tmPw, const __grid_constant__ CUtensorMap tmPx,
                     const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const GradArgs a) {
  using C = GradCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf_bar[i], 1);
      mbar_init(&acce_bar[i], 2 * kGradEpiWarps);  // both CTAs' epilogue warps
    }
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_cg<2>(&tmem_base_sh, C::TMEM_COLS);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are initialised before any cross-CTA arrive or copy
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tmem = tmem_base_sh;
  const uint64_t tmo = a.timeout_ns;
  const uint32_t full_lead0 = mapa_shared(smem_u32(&full_bar[0]), 0);
  const uint32_t acce_lead0 = mapa_shared(smem_u32(&acce_bar[0]), 0);
  const int pair = (int)cluster_id_x(), pairs = (int)nclusters_x();

  auto give_up = [&](int code) {
    abort_sh = 1;
    if (a.err) atomicExch(a.err, code);
  };

  GradUnit u;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    const bool issuer = elect_one();
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_par = 0;
    bool ok = true;
    for (int i = 0; ok && grad_unit(a, pair, pairs, i, BN, u); ++i) {
      const int m = u.m0 + (int)rank * 128, n = u.n0 + (int)rank * (BN / 2);
      for (int kb = u.kb0; kb < u.kb1; ++kb) {
        if (!mbar_wait_warp(&empty_bar[stage], phase ^ 1u, &abort_sh, tmo)) {
          if (issuer) give_up(1);
          ok = false;
          break;
        }
        if (issuer) {
          uint8_t* st = smem + (size_t)stage * C::STAGE;
          const uint32_t fb = full_lead0 + 8u * (uint32_t)stage;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], (uint32_t)(2 * C::STAGE));
          if (u.dw) {
            const int t = kb * kGradKb;
            tma_load_3d_pair(st, &tmPw, fb, m, u.z, t);
            tma_load_3d_pair(st + C::RUN, &tmPw, fb, m + 64, u.z, t);
#pragma unroll
            for (int j = 0; j < C::NB; ++j)
              tma_load_3d_pair(st + C::A_BYTES + j * C::RUN, &tmX, fb, n + 64 * j, t, 0);
          } else {
            const int z = kb >= a.kb_half ? 1 : 0, f = (kb - z * a.kb_half) * kGradKb;
            tma_load_3d_pair(st, &tmPx, fb, f, z, m);
#pragma unroll
            for (int j = 0; j < C::NB; ++j)
              tma_load_3d_pair(st + C::A_BYTES + j * C::RUN, &tmW, fb, n + 64 * j, f, z);
          }
        }
        armed |= 1u << stage;
        armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (leader)  // drain: both CTAs' copies have landed (the peer is held by the cluster barrier below)
      for (int i = 0; i < C::STAGES; ++i)
        if ((armed >> i) & 1u) mbar_wait_warp(&full_bar[i], (armed_par >> i) & 1u, &abort_sh, tmo);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (leader) {
      const bool issuer = elect_one();
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int i = 0; ok && grad_unit(a, pair, pairs, i, BN, u); ++i) {
        const uint32_t idesc = u.dw ? grad_idesc<DT, BN>(true) : grad_idesc<DT, BN>(false);
        // per MMA (16 summed elements): 32 bytes along a K-major row, 16 rows of an MN-major run
        const uint64_t a_step = u.dw ? (16u * 128u) >> 4 : 32u >> 4, b_step = (16u * 128u) >> 4;
        for (int r0 = u.kb0; ok && r0 < u.kb1; r0 += kRunKb) {
          const int r1 = min(u.kb1, r0 + kRunKb);
          if (!mbar_wait_warp(&acce_bar[acc], acc_phase ^ 1u, &abort_sh, tmo)) {
            if (issuer) give_up(2);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
          for (int kb = r0; kb < r1; ++kb) {
            if (!mbar_wait_warp(&full_bar[stage], phase, &abort_sh, tmo)) {
              if (issuer) give_up(3);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(smem + (size_t)stage * C::STAGE), b_addr = a_addr + C::A_BYTES;
            const uint64_t ad0 = u.dw ? sdesc_sw128_mn(a_addr, C::RUN) : sdesc_sw128(a_addr);
            const uint64_t bd0 = sdesc_sw128_mn(b_addr, C::RUN);
            if (issuer) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_pair<1>(d_tmem, ad0 + a_step * j, bd0 + b_step * j, idesc, (kb > r0 || j > 0) ? 1u : 0u);
              tc_commit_pair(&empty_bar[stage], (uint16_t)3);
            }
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (issuer) tc_commit_pair(&accf_bar[acc], (uint16_t)3);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (issuer) tc_commit_pair(&drain_bar, (uint16_t)3);
    }
    mbar_wait_warp(&drain_bar, 0, &abort_sh, tmo);  // every MMA of this pair has completed
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    constexpr int OT = DT == DT_F16 ? OUT_F16 : OUT_BF16;
    const int ew = warp - 2, lq = warp & 3, part = ew >> 2;
    uint8_t* buf = smem + (size_t)C::STAGES * C::STAGE + (size_t)ew * C::EPI_BUF;
    if (a.dbias)  // while the first tile is summed
      for (int c = ((int)blockIdx.x * kGradEpiWarps + ew) * 4; c < 2 * a.F; c += (int)gridDim.x * kGradEpiWarps * 4)
        dbias_columns(a.part, 2 * a.F, a.row_blocks, c, lane, a.dbias);
    // this warp's columns of the runs so far, [WCOLS][32 lanes]: a thread reads back what it wrote
    float* run = a.runs + ((size_t)(2 * pair + (int)rank) * kGradEpiWarps + ew) * (C::WCOLS * 32) + lane;
    [[maybe_unused]] float undo = 1.0f;
    if constexpr (DT == DT_F16) undo = __ldcg(a.undo);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int i = 0; ok && grad_unit(a, pair, pairs, i, BN, u); ++i) {
      for (int k0 = u.kb0; k0 < u.kb1; k0 += kRunKb) {
        const bool first = k0 == u.kb0, last = k0 + kRunKb >= u.kb1;
        if (!mbar_wait_warp(&accf_bar[acc], acc_phase, &abort_sh, tmo)) {
          if (lane == 0) give_up(4);
          ok = false;
          break;
        }
        tc_fence_after();
        const int r0 = (int)rank * 128 + lq * 32, c0 = part * C::WCOLS;
        const int row0 = u.m0 + r0, col0 = u.n0 + c0;
        const int rows = min(32, (u.dw ? a.F : a.T) - row0);
        uint8_t* out = static_cast<uint8_t*>(u.dw ? a.dW : a.dX) +
                       ((int64_t)(u.dw ? u.z * a.F : 0) + row0) * a.k * 2;
        float* fp32 = a.partial + ((size_t)max(u.slot, 0) * 256 + r0) * BN + c0;
        const uint32_t taddr = tmem + ((uint32_t)(lq * 32) << 16) + (uint32_t)(acc * BN + c0);
#pragma unroll 1
        for (int c = 0; c < C::WCOLS; c += 64) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            __syncwarp();
            tmem_ld32(taddr + (uint32_t)(c + 32 * h), *reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_wait_ld();
            if (h == 1 && c + 64 == C::WCOLS) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(acce_lead0 + 8u * (uint32_t)acc);
            }
            float* so_far = run + (c + 32 * h) * 32;
            if (!first) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += __ldcg(so_far + j * 32);
            }
            if (!last) {
#pragma unroll
              for (int j = 0; j < 32; ++j) __stcg(so_far + j * 32, v[j]);
              continue;
            }
            if (u.slot >= 0) {
              stage_row<OUT_F32, 128, 32>(buf, (uint32_t)lane, 0, v);
              __syncwarp();
              stage_flush<128, 4>(buf, reinterpret_cast<uint8_t*>(fp32 + c + 32 * h), (int64_t)BN * 4, 32, 128, true, lane);
            } else {
              if constexpr (DT == DT_F16) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= undo;
              }
              stage_row<OT, 128, 32>(buf, (uint32_t)lane, (uint32_t)(4 * h), v);
            }
          }
          __syncwarp();
          if (last && u.slot < 0 && rows > 0 && col0 + c < a.k)
            stage_flush<128, 2>(buf, out + (int64_t)(col0 + c) * 2, (int64_t)a.k * 2, rows, min(64, a.k - col0 - c) * 2,
                                true, lane);
          __syncwarp();
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every remote arrive and copy of the pair is done before either CTA frees anything
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<2>(tmem, C::TMEM_COLS);
  }
}

// Adds up the parts of split tiles, in order, and rounds once.  A block takes eight
// rows of one tile (blockIdx.y), a warp a row of it, a lane four columns at a time;
// eight parts' loads are in flight.
template <int DT, int BN>
__global__ void __launch_bounds__(256) grad_join_kernel(const GradArgs a) {
  constexpr int OT = DT == DT_F16 ? OUT_F16 : OUT_BF16;
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = a.side[0].splits > 1 ? a.side[0].tiles : 0;  // split tiles of side 0 come first
  const int s = (int)blockIdx.y >= t0 ? 1 : 0, tile = (int)blockIdx.y - s * t0;
  const GradSide& g = a.side[s];
  const int first = g.slot0 + tile * g.splits;
  const int nt = tile % g.n_nt, mt = tile / g.n_nt, z = g.dw ? mt / g.n_mt : 0;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), m = (g.dw ? mt % g.n_mt : mt) * 256 + row;
  if (m >= (g.dw ? a.F : a.T)) return;
  uint16_t* out = static_cast<uint16_t*>(g.dw ? a.dW : a.dX) + ((int64_t)(z * a.F) + m) * a.k;
  [[maybe_unused]] float undo = 1.0f;
  if constexpr (DT == DT_F16) undo = __ldcg(a.undo);
  for (int c = (threadIdx.x & 31) * 4; c < BN && nt * BN + c < a.k; c += 128) {
    const float* src = a.partial + ((size_t)first * 256 + row) * BN + c;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int p = 0; p < g.splits; ++p) {
      const float4 w = *reinterpret_cast<const float4*>(src + (size_t)p * 256 * BN);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    if constexpr (DT == DT_F16) {
      v.x *= undo;
      v.y *= undo;
      v.z *= undo;
      v.w *= undo;
    }
    *reinterpret_cast<uint2*>(out + nt * BN + c) = make_uint2(pack_pair<OT>(v.x, v.y), pack_pair<OT>(v.z, v.w));
  }
}

struct GradMaps {
  CUtensorMap pw, px, x, w;
};

template <int DT, int BN>
cudaError_t launch_grad_t(int grid, const GradMaps& m, const GradArgs& a, cudaStream_t s) {
  auto kern = grad_pair_kernel<DT, BN>;
  static std::atomic<uint64_t> opted{0};
  cudaError_t e = smem_opt_in(kern, GradCfg<BN>::SMEM, opted);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)(2 * grid)), kGradThreads, GradCfg<BN>::SMEM, s, 0, m.pw, m.px, m.x, m.w, a);
  if (e != cudaSuccess) return e;
  const int tiles = (a.side[0].splits > 1 ? a.side[0].tiles : 0) + (a.side[1].splits > 1 ? a.side[1].tiles : 0);
  return tiles ? launch_pdl(grad_join_kernel<DT, BN>, dim3(32, (unsigned)tiles), 256, 0, s, 0, a) : cudaSuccess;
}

// Rows per block: eight a warp, or two when that would leave SMs without a block
// (1379 x 2 x 2051 with the bias: 18.6 us with 16 rows a warp, 11.1 with two).
int dp_block_rows(int64_t T, int64_t F, int sms) {
  const int64_t col_blocks = (F + kDpCols - 1) / kDpCols;
  return (T + 63) / 64 * col_blocks >= 4 * sms ? 64 : 16;
}

template <int DT>
cudaError_t launch_dp(bool vec, const void* P, const void* dY, int T, int F, int pitch, int act, void* dp, float* part,
                      uint32_t* peak, float* undo, const UnpackArgs& un, int sms, cudaStream_t s) {
  const int rows = dp_block_rows(T, F, sms), col_blocks = (F + kDpCols - 1) / kDpCols;
  const int64_t blocks = (int64_t)((T + rows - 1) / rows) * col_blocks;
  const uint16_t *p = static_cast<const uint16_t*>(P), *y = static_cast<const uint16_t*>(dY);
  uint16_t* o = static_cast<uint16_t*>(dp);
  auto kern = vec ? (part ? gated_dp_kernel<DT, true, true> : gated_dp_kernel<DT, true, false>)
                  : (part ? gated_dp_kernel<DT, false, true> : gated_dp_kernel<DT, false, false>);
  cudaError_t e = launch_pdl(kern, dim3((unsigned)(blocks + un.blocks)), 32 * kDpWarps, 0, s, 0, p, y, T, F, pitch, act, o,
                             part, peak, rows, col_blocks, un);
  if constexpr (DT == DT_F16) {
    if (e == cudaSuccess && peak)
      e = launch_pdl(vec ? gated_dp_scale_kernel<true> : gated_dp_scale_kernel<false>,
                     dim3((unsigned)std::min<int64_t>(blocks, 4 * sms)), 32 * kDpWarps, 0, s, 0, p, y, T, F, pitch, act, o,
                     (const uint32_t*)peak, (int)blocks, rows, col_blocks, undo);
  }
  return e;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Shares the units of two products out over at most `pairs` CTA pairs: side 0 (the
// longer units) goes round the pairs, side 1 on top so that the fullest pair has
// the least to do.  Returns that pair's stages, with a fixed part per unit.
int64_t share_out(const GradSide& x, const GradSide& y, int pairs, GradArgs* a, int* grid) {
  constexpr int kFixed = 6;  // a unit's fill and drain, in stages
  const bool x_first = x.per_split >= y.per_split;
  a->side[0] = x_first ? x : y;
  a->side[1] = x_first ? y : x;
  const int64_t n0 = (int64_t)a->side[0].tiles * a->side[0].splits, n1 = (int64_t)a->side[1].tiles * a->side[1].splits;
  const int64_t c0 = a->side[0].per_split + kFixed, c1 = a->side[1].per_split + kFixed;
  *grid = (int)std::min<int64_t>(n0 + n1, pairs);
  const int64_t q = n0 / *grid;
  a->hi = (int)(n0 % *grid);
  // the lowest level (in stages) at which every unit of side 1 finds room
  auto room = [&](int64_t level, int64_t* lo, int64_t* hi) {
    *lo = std::max<int64_t>(0, (level - q * c0) / c1);
    *hi = a->hi ? std::max<int64_t>(0, (level - (q + 1) * c0) / c1) : *lo;
    return *lo * (*grid - a->hi) + *hi * a->hi >= n1;
  };
  int64_t lo = 0, hi = 0, below = (n0 * c0 + n1 * c1) / *grid - 1, level = below + c0 + c1 + 1;
  while (level - below > 1) {  // room at `level` (the average and a unit of each side more), none at `below`
    const int64_t mid = (below + level) / 2;
    (room(mid, &lo, &hi) ? level : below) = mid;
  }
  room(level, &lo, &hi);
  a->lo_units = (int)lo;
  a->hi_units = (int)hi;
  return std::max(q * c0 + lo * c1, a->hi ? (q + 1) * c0 + hi * c1 : 0);
}

// The launch for tiles bn columns wide: its stages (share_out), or -1 when there
// are too many tiles.
int64_t plan_grad(int64_t F, int64_t k, int64_t T, bool want_dx, bool want_dw, int bn, int pairs, bool may_cut,
                  GradArgs* a, int* grid) {
  const int n_nt = (int)((k + bn - 1) / bn);
  a->F = (int)F;
  a->T = (int)T;
  a->k = (int)k;
  a->kb_half = (int)((F + kGradKb - 1) / kGradKb);
  GradSide sw{}, sx{};
  sw.dw = 1;
  sw.n_nt = sx.n_nt = n_nt;
  sw.n_mt = (int)((F + 255) / 256);
  sw.n_kb = (int)((T + kGradKb - 1) / kGradKb);
  sx.n_mt = (int)((T + 255) / 256);
  sx.n_kb = 2 * a->kb_half;
  const int64_t w_tiles = want_dw ? 2 * (int64_t)sw.n_mt * n_nt : 0, x_tiles = want_dx ? (int64_t)sx.n_mt * n_nt : 0;
  if (w_tiles > INT32_MAX / 2 || x_tiles > INT32_MAX / 2) return -1;
  sw.tiles = (int)w_tiles;
  sx.tiles = (int)x_tiles;
  sw.splits = sx.splits = 1;
  sw.per_split = sw.n_kb;
  sx.per_split = sx.n_kb;
  int64_t cost = share_out(sw, sx, pairs, a, grid);
  if (!may_cut) return cost;

  // Cut long sums into parts of at most `len` stages where that leaves the fullest
  // pair less to do.  Joining the parts (fp32 tiles out to L2, another launch)
  // costs about kJoin stages.  The workspace holds a partial tile per pair.
  constexpr int kJoin = 24;
  const int longest = std::max(sw.tiles ? sw.n_kb : 0, sx.tiles ? sx.n_kb : 0);
  const int64_t sum = (int64_t)sw.tiles * sw.n_kb + (int64_t)sx.tiles * sx.n_kb;
  for (int len = 8; len < longest && std::max<int64_t>(len, sum / pairs) + kJoin < cost; len += len / 2) {
    GradSide side[2] = {sw, sx};
    int64_t parts = 0;
    for (GradSide& g : side) {
      g.splits = g.tiles ? (g.n_kb + len - 1) / len : 1;
      g.per_split = (g.n_kb + g.splits - 1) / g.splits;
      g.splits = (g.n_kb + g.per_split - 1) / g.per_split;  // no part is empty
      g.slot0 = (int)parts;
      if (g.splits > 1) parts += (int64_t)g.tiles * g.splits;
      if (parts > pairs) break;
    }
    if (parts > pairs || parts == 0) continue;
    GradArgs c = *a;
    int g = 0;
    const int64_t level = share_out(side[0], side[1], pairs, &c, &g) + kJoin;
    if (level < cost) {
      cost = level;
      *a = c;
      *grid = g;
    }
  }
  return cost;
}

// Workspace: dp, the masked dense weight, the row blocks' column sums, fp16: the factor
// that undoes dp's scaling and the blocks' largest |dp|, partial tiles of cut sums (one
// per pair at most), and a tile per pair for sums of several runs.
struct GradWs {
  int64_t pitch, dp, wm, part, undo, peak, partial, runs, total;
  GradWs(const nm_handle* h, int64_t T) {
    const int sms = num_sms(h->device);
    const int64_t F = h->n_out / 2, pairs = sms / 2;
    pitch = (F + 63) / 64 * 64;  // whole 128-byte lines: a 128-byte box row then touches one
    dp = 0;
    wm = dp + align256(T * 2 * pitch * 2);
    part = wm + align256(h->n_out * h->k * 2);
    const int64_t rows = dp_block_rows(T, F, sms);
    undo = part + align256((T + rows - 1) / rows * h->n_out * 4);
    peak = undo + 256;
    partial = h->dt == DT_F16 ? peak + align256((T + rows - 1) / rows * ((F + kDpCols - 1) / kDpCols) * 4) : undo;
    // with more 128-wide tiles than twice the pairs on both sides nothing is cut
    const int64_t n_nt = (h->k + 127) / 128, tiles = std::min(2 * ((F + 255) / 256), (T + 255) / 256) * n_nt;
    const int64_t tile_bytes = pairs * 256 * 256 * 4, longest = std::max(T, 2 * ((F + kGradKb - 1) / kGradKb) * kGradKb);
    runs = partial + (tiles <= 2 * pairs ? tile_bytes : 0);
    total = runs + (longest > (int64_t)kRunKb * kGradKb ? tile_bytes : 0);
  }
};

int forced_grad_bn() {  // tests and sweeps
  const char* v = getenv("NMSPMM_FORCE_GRAD_BN");
  return v && *v ? atoi(v) : 0;
}

// The tile width with the lower estimate of the fullest pair's work, and its
// launch.  A stage of a 256-wide tile takes 1.45 times a 128-wide one's (0.33
// against 0.23 us over full waves, 0.28 against 0.19 when few tiles run; the
// narrower tile moves 24 KB a stage and SM against 32 KB for half the products).
// The choice is a function of the shape alone; a thread's last one is kept, since a
// training step asks for the same again and again.
nm_status choose_grad(int64_t F, int64_t k, int64_t T, bool want_dx, bool want_dw, int pairs, GradArgs* a, int* grid,
                      int* bn) {
  struct Key {
    int64_t F, k, T;
    int want, pairs, forced, whole;
    bool operator==(const Key& o) const {
      return F == o.F && k == o.k && T == o.T && want == o.want && pairs == o.pairs && forced == o.forced &&
             whole == o.whole;
    }
  };
  struct Choice {
    Key key{};
    GradArgs a{};
    int grid = 0, bn = 0;
  };
  static thread_local Choice last;
  const int forced = forced_grad_bn();
  const char* split = getenv("NMSPMM_GRAD_SPLIT");  // 0: no split (tests and sweeps)
  const Key key{F, k, T, (want_dx ? 1 : 0) + (want_dw ? 2 : 0), pairs, forced, split && split[0] == '0'};
  if (last.bn && last.key == key) {
    *a = last.a;
    *grid = last.grid;
    *bn = last.bn;
    return NM_OK;
  }
  *bn = 0;
  double best = 1e300;
  for (int w : {256, 128}) {
    if (forced && w != forced) continue;
    GradArgs c{};
    int g = 0;
    const int64_t level = plan_grad(F, k, T, want_dx, want_dw, w, pairs, !key.whole, &c, &g);
    if (level < 0) return fail(NM_ERR_UNSUPPORTED, "T x k too large");
    const double cost = (double)level * (w == 256 ? 1.45 : 1.0);
    if (cost < best) {
      best = cost;
      *a = c;
      *bn = w;
      *grid = g;
    }
  }
  if (!*bn) return fail(NM_ERR_INVALID, "NMSPMM_FORCE_GRAD_BN must be 128 or 256");
  last.key = key;
  last.a = *a;
  last.grid = *grid;
  last.bn = *bn;
  return NM_OK;
}

nm_status check_grad(const nm_handle* h, int64_t T) {
  nm_status st = check_handle(h);
  if (st != NM_OK) return st;
  if (!h->gated || h->mx) return fail(NM_ERR_INVALID, "nm_gated_backward needs a handle made by nm_compress_gated");
  if (h->dt == DT_I8) return fail(NM_ERR_UNSUPPORTED, "gradients are for FP16 and BF16 handles only");
  if (T < 0) return fail(NM_ERR_INVALID, "T must be >= 0 (got %lld)", (long long)T);
  // tokens, row blocks and stages are counted in 32 bits, with room to spare
  if (T > (int64_t(1) << 26)) return fail(NM_ERR_UNSUPPORTED, "T above 2^26");
  return NM_OK;
}

// A 16-bit tensor of three dimensions (strides in elements).
nm_status map16(CUtensorMap* m, int dt, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2,
                int b0, int b1, int b2, CUtensorMapSwizzle swizzle) {
  const uint64_t dims[3] = {(uint64_t)d0, (uint64_t)d1, (uint64_t)d2};
  const uint64_t strides[2] = {(uint64_t)s1 * 2, (uint64_t)s2 * 2};
  const uint32_t box[3] = {(uint32_t)b0, (uint32_t)b1, (uint32_t)b2};
  return encode_map(m, dt == DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
                    strides, box, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace
}  // namespace nm

using namespace nm;

extern "C" {

nm_status nm_gated_backward_workspace(const nm_handle* h, int64_t T, size_t* bytes) {
  clear_error();
  nm_status st = check_grad(h, T);
  if (st != NM_OK) return st;
  if (!bytes) return fail(NM_ERR_INVALID, "null output");
  *bytes = (size_t)GradWs(h, T).total;
  return NM_OK;
}

nm_status nm_gated_backward_plan_for_shape(int64_t n_ff, int64_t k, int64_t T, int want_dx, int want_dw, int sms,
                                           nm_grad_plan_info* out) {
  clear_error();
  if (!out) return fail(NM_ERR_INVALID, "null output");
  if (n_ff <= 0 || k <= 0 || T <= 0 || sms < 2) return fail(NM_ERR_INVALID, "bad shape or SM count");
  if (!want_dx && !want_dw) return fail(NM_ERR_INVALID, "nothing to compute");
  if (n_ff > (1 << 23) || k > (1 << 24) || T > (int64_t(1) << 26)) return fail(NM_ERR_UNSUPPORTED, "shape too large");
  GradArgs a{};
  int grid = 0, bn = 0;
  nm_status st = choose_grad(n_ff, k, T, want_dx != 0, want_dw != 0, sms / 2, &a, &grid, &bn);
  if (st != NM_OK) return st;
  *out = nm_grad_plan_info{};
  out->bn = bn;
  out->grid = grid;
  for (const GradSide& g : a.side) {
    if (!g.tiles) continue;
    (g.dw ? out->splits_dw : out->splits_dx) = g.splits;
    (g.dw ? out->runs_dw : out->runs_dx) = (g.per_split + kRunKb - 1) / kRunKb;
  }
  // every stage of every tile is some pair's, once; a cut tile's parts have slots of their own
  int64_t stages = 0, want = (int64_t)a.side[0].tiles * a.side[0].n_kb + (int64_t)a.side[1].tiles * a.side[1].n_kb;
  int64_t slots = 0, slot_sum = 0;
  for (int pair = 0; pair < grid; ++pair) {
    int64_t mine = 0;
    GradUnit u;
    for (int i = 0; grad_unit(a, pair, grid, i, bn, u); ++i) {
      mine += u.kb1 - u.kb0;
      if (u.slot >= 0) {
        ++slots;
        slot_sum += u.slot;
      }
    }
    stages += mine;
    out->stages = std::max<int64_t>(out->stages, mine);
  }
  out->complete = stages == want && slot_sum == slots * (slots - 1) / 2 && slots <= sms / 2;
  return NM_OK;
}

nm_status nm_gated_backward(const nm_handle* h, const void* X, const void* P, const void* dY, int64_t T, nm_act act,
                            void* dX, void* dW, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  nm_status st = check_grad(h, T);
  if (st != NM_OK) return st;
  if ((int)act < 0 || (int)act > (int)NM_ACT_RELU) return fail(NM_ERR_INVALID, "unknown activation %d", (int)act);
  if (!dX && !dW && !dbias) return fail(NM_ERR_INVALID, "nothing to compute: dX, dW and dbias are null");
  if (h->k % 8 != 0) return fail(NM_ERR_UNSUPPORTED, "k must be a multiple of 8 (k=%lld)", (long long)h->k);
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t F = h->n_out / 2;
  const size_t pbytes = (size_t)T * h->n_out * 2, ybytes = (size_t)T * F * 2, xbytes = (size_t)T * h->k * 2;
  const size_t wbytes = (size_t)h->n_out * h->k * 2, bbytes = (size_t)h->n_out * 4;
  if (!aligned(dX, 16) || !aligned(dW, 16) || !aligned(dbias, 16) || !aligned(X, 16) || !aligned(P, 16) ||
      !aligned(dY, 16) || !aligned(ws, 16))
    return fail(NM_ERR_INVALID, "all pointers must be 16-byte aligned");
  if (T == 0) {
    cudaError_t e = cudaSuccess;
    if (dW) e = cudaMemsetAsync(dW, 0, wbytes, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, bbytes, s);
    return e == cudaSuccess ? NM_OK : cuda_fail(e, "clear the gradients");
  }
  if (!P || !dY || (dW && !X)) return fail(NM_ERR_INVALID, "null P, dY or X");
  const GradWs lay(h, T);
  if (!ws || ws_bytes < (size_t)lay.total)
    return fail(NM_ERR_INVALID, "the workspace holds %zu bytes, %lld are needed", ws ? ws_bytes : (size_t)0,
                (long long)lay.total);
  {
    const void* buf[7] = {dX, dW, dbias, ws, P, dY, dW ? X : nullptr};
    const size_t len[7] = {xbytes, wbytes, bbytes, (size_t)lay.total, pbytes, ybytes, xbytes};
    for (int i = 0; i < 4; ++i)  // what is written shares nothing with the rest
      for (int j = i + 1; j < 7; ++j)
        if (buf[i] && buf[j] && overlaps(buf[i], len[i], buf[j], len[j]))
          return fail(NM_ERR_INVALID, "outputs, workspace and inputs overlap");
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  void* dp = base + lay.dp;
  float* part = dbias ? reinterpret_cast<float*>(base + lay.part) : nullptr;
  const int sms = num_sms(h->device), rows = dp_block_rows(T, F, sms), row_blocks = (int)((T + rows - 1) / rows);
  UnpackArgs un{};
  if (dX) {
    un.bpack = h->d_bpack;
    un.Wm = reinterpret_cast<uint16_t*>(base + lay.wm);
    un.K = h->k;
    un.units = h->n_out * ((h->k + 15) / 16);
    un.img = h->img;
    un.n_kb = h->n_kb;
    un.n_ff = (int)F;
    un.blocks = (int)((un.units + 32 * kDpWarps - 1) / (32 * kDpWarps));
  }
  if ((int64_t)row_blocks * ((F + kDpCols - 1) / kDpCols) + un.blocks > INT32_MAX)
    return fail(NM_ERR_UNSUPPORTED, "T x n_ff too large");
  GradArgs a{};
  int bn = 0, grid = 0;
  if ((dX || dW) && (st = choose_grad(F, h->k, T, dX != nullptr, dW != nullptr, sms / 2, &a, &grid, &bn)) != NM_OK)
    return st;
  if ((a.side[0].splits > 1 || a.side[1].splits > 1) && lay.partial == lay.runs)
    return fail(NM_ERR_INVALID, "the workspace has no room for partial tiles");
  cudaError_t e = cudaSuccess;
  const bool vec = F % 8 == 0;  // every row starts on 16 bytes
  float* undo = reinterpret_cast<float*>(base + lay.undo);
  uint32_t* peak = h->dt == DT_F16 && (dX || dW) ? reinterpret_cast<uint32_t*>(base + lay.peak) : nullptr;
  e = h->dt == DT_F16
          ? launch_dp<DT_F16>(vec, P, dY, (int)T, (int)F, (int)lay.pitch, (int)act, dp, part, peak, undo, un, sms, s)
          : launch_dp<DT_BF16>(vec, P, dY, (int)T, (int)F, (int)lay.pitch, (int)act, dp, part, peak, undo, un, sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "launch the gradient of the output stage");

  if (dX || dW) {
    a.partial = reinterpret_cast<float*>(base + lay.partial);
    a.runs = reinterpret_cast<float*>(base + lay.runs);
    a.dW = dW;
    a.dX = dX;
    a.undo = undo;
    a.part = part;
    a.dbias = dbias;
    a.row_blocks = row_blocks;
    a.err = h->d_err;
    a.timeout_ns = 1000000000ull;

    GradMaps m;
    const int dt = h->dt;
    const void* wm = base + lay.wm;
    const auto k128 = CU_TENSOR_MAP_SWIZZLE_128B;
    st = map16(&m.pw, dt, dp, F, 2, T, lay.pitch, 2 * lay.pitch, 64, 1, 64, k128);
    if (st == NM_OK) st = map16(&m.px, dt, dp, F, 2, T, lay.pitch, 2 * lay.pitch, 64, 1, 128, k128);
    m.x = m.w = m.pw;  // of a product that is not asked for: never read
    if (st == NM_OK && dW) st = map16(&m.x, dt, X, h->k, T, 1, h->k, h->k * T, 64, 64, 1, k128);
    if (st == NM_OK && dX) st = map16(&m.w, dt, wm, h->k, F, 2, h->k, h->k * F, 64, 64, 1, k128);
    if (st != NM_OK) return st;
    e = dt == DT_F16 ? (bn == 256 ? launch_grad_t<DT_F16, 256>(grid, m, a, s) : launch_grad_t<DT_F16, 128>(grid, m, a, s))
                     : (bn == 256 ? launch_grad_t<DT_BF16, 256>(grid, m, a, s)
                                  : launch_grad_t<DT_BF16, 128>(grid, m, a, s));
    if (e != cudaSuccess) return cuda_fail(e, "launch the gradient products");
  }
  if (dbias && !dX && !dW) {
    e = launch_pdl(dbias_kernel, dim3((unsigned)((h->n_out + 15) / 16)), 128, 0, s, 0, (const float*)part,
                   (int)h->n_out, row_blocks, dbias);
    if (e != cudaSuccess) return cuda_fail(e, "launch the bias gradient");
  }
  return NM_OK;
}

}  // extern "C"

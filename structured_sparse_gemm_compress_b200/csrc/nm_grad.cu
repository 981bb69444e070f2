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

#include "nm_act.cuh"
#include "nm_api_internal.h"
#include "nm_device.cuh"
#include "nm_launch.cuh"
#include "nm_stage.cuh"

namespace nm {
namespace {

// ------------------------------------------------------------------ dp and dbias

constexpr int kDpCols = 256;  // columns of each half per block
constexpr int kDpRows = 128;  // rows per block
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
    if (f0 + lane * 8 < F) q = __ldg(reinterpret_cast<const uint4*>(row + f0 + lane * 8));
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
      v[j] = f < F ? to_f32<DT>(__ldg(row + f)) : 0.0f;
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

// One pass over P and dY: dp [T][2][pitch] in the handle's type (rounded for the
// tensor core; columns n_ff .. pitch are never read) and, with `part`, the fp32
// column sums of this block's rows ([row block][2][n_ff]), each warp's rows in
// ascending order, the warps in order.  Memory bound.
// BIAS is its own instance: the sums' registers cost the plain one a third of its
// warps.
template <int DT, bool VEC, bool BIAS>
__global__ void __launch_bounds__(32 * kDpWarps, BIAS ? 3 : 4)
    gated_dp_kernel(const uint16_t* __restrict__ P, const uint16_t* __restrict__ dY, int T, int F, int pitch, int act,
                    uint16_t* __restrict__ dp, float* __restrict__ part) {
  __shared__ float sums[BIAS ? kDpWarps : 1][2][kDpCols];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int f0 = blockIdx.x * kDpCols, t0 = blockIdx.y * kDpRows;
  const int t1 = min(T, t0 + kDpRows);
  float sg[8] = {}, su[8] = {};
  for (int t = t0 + warp; t < t1; t += kDpWarps) {
    const uint16_t* prow = P + (size_t)t * 2 * F;
    float g[8], u[8], dy[8];
    dp_load<DT, VEC>(prow, f0, F, lane, g);
    dp_load<DT, VEC>(prow + F, f0, F, lane, u);
    dp_load<DT, VEC>(dY + (size_t)t * F, f0, F, lane, dy);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, d;
      act_slope(g[j], act, a, d);
      g[j] = __fmul_rn(__fmul_rn(dy[j], u[j]), d);
      u[j] = __fmul_rn(dy[j], a);
      if constexpr (BIAS) {
        sg[j] += g[j];
        su[j] += u[j];
      }
    }
    uint16_t* out = dp + (size_t)t * 2 * pitch;
    dp_store<DT, VEC>(out, f0, F, lane, g);
    dp_store<DT, VEC>(out + pitch, f0, F, lane, u);
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
      if (f0 + c < F) part[((size_t)blockIdx.y * 2 + z) * F + f0 + c] = s;
    }
  }
}

// dbias [2 n_ff]: the row blocks' sums, eight interleaved runs of them per column, the runs in order.
__global__ void __launch_bounds__(256) dbias_kernel(const float* __restrict__ part, int n, int blocks,
                                                    float* __restrict__ dbias) {
  __shared__ float sums[8][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < n)
    for (int b = run; b < blocks; b += 8) s += part[(size_t)b * n + c];
  sums[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < n) {
#pragma unroll
    for (int r = 1; r < 8; ++r) s += sums[r][lane];
    dbias[c] = s;
  }
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
constexpr int kGradKb = 64;
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
};

struct GradArgs {
  GradSide side[2];
  int hi;                  // pairs with one more tile of side 0 than the others
  int hi_tiles, lo_tiles;  // tiles of side 1 for those pairs, and for the others
  int F, T, k;
  int kb_half;       // dX: stages per half of 2 n_ff
  void *dW, *dX;
  int* err;
  unsigned long long timeout_ns;
};

struct GradUnit {
  int dw, m0, n0, z, n_kb;
};

// The i-th unit of this pair; false when there is none.  Side 0's tiles go round
// the pairs; `hi` pairs get one more of them than the others.  Side 1's: first
// lo_tiles - hi_tiles rounds over the other pairs alone, then hi_tiles rounds
// over all (hi_tiles <= lo_tiles), the last round cut off at the end of the list.
__device__ __forceinline__ bool grad_unit(const GradArgs& a, int pair, int pairs, int i, int bn, GradUnit& u) {
  const int q = a.side[0].tiles / pairs + (pair < a.hi ? 1 : 0);
  int s = 0, tile;
  if (i < q) {
    tile = i * pairs + pair;
  } else {
    s = 1;
    int r = i - q;
    const int extra = a.lo_tiles - a.hi_tiles, lo_pairs = pairs - a.hi;
    if (pair >= a.hi) {
      if (r < extra) {
        tile = r * lo_pairs + (pair - a.hi);
      } else {
        r -= extra;
        if (r >= a.hi_tiles) return false;
        tile = extra * lo_pairs + r * pairs + (pair - a.hi);
      }
    } else {
      if (r >= a.hi_tiles) return false;
      tile = extra * lo_pairs + r * pairs + lo_pairs + pair;
    }
    if (tile >= a.side[1].tiles) return false;
  }
  const GradSide& g = a.side[s];
  const int nt = tile % g.n_nt, mt = tile / g.n_nt;
  u.dw = g.dw;
  u.n_kb = g.n_kb;
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
      for (int kb = 0; kb < u.n_kb; ++kb) {
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
        if (!mbar_wait_warp(&acce_bar[acc], acc_phase ^ 1u, &abort_sh, tmo)) {
          if (issuer) give_up(2);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
        const uint32_t idesc = u.dw ? grad_idesc<DT, BN>(true) : grad_idesc<DT, BN>(false);
        // per MMA (16 summed elements): 32 bytes along a K-major row, 16 rows of an MN-major run
        const uint64_t a_step = u.dw ? (16u * 128u) >> 4 : 32u >> 4, b_step = (16u * 128u) >> 4;
        for (int kb = 0; kb < u.n_kb; ++kb) {
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
              tc_mma_pair<1>(d_tmem, ad0 + a_step * j, bd0 + b_step * j, idesc, (kb > 0 || j > 0) ? 1u : 0u);
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
      if (issuer) tc_commit_pair(&drain_bar, (uint16_t)3);
    }
    mbar_wait_warp(&drain_bar, 0, &abort_sh, tmo);  // every MMA of this pair has completed
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    constexpr int OT = DT == DT_F16 ? OUT_F16 : OUT_BF16;
    const int ew = warp - 2, lq = warp & 3, part = ew >> 2;
    uint8_t* buf = smem + (size_t)C::STAGES * C::STAGE + (size_t)ew * C::EPI_BUF;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int i = 0; grad_unit(a, pair, pairs, i, BN, u); ++i) {
      if (!mbar_wait_warp(&accf_bar[acc], acc_phase, &abort_sh, tmo)) {
        if (lane == 0) give_up(4);
        break;
      }
      tc_fence_after();
      const int row0 = u.m0 + (int)rank * 128 + lq * 32, col0 = u.n0 + part * C::WCOLS;
      const int rows = min(32, (u.dw ? a.F : a.T) - row0);
      uint8_t* out = static_cast<uint8_t*>(u.dw ? a.dW : a.dX) +
                     ((int64_t)(u.dw ? u.z * a.F : 0) + row0) * a.k * 2;
      const uint32_t taddr = tmem + ((uint32_t)(lq * 32) << 16) + (uint32_t)(acc * BN + part * C::WCOLS);
#pragma unroll 1
      for (int c = 0; c < C::WCOLS; c += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(taddr + (uint32_t)(c + 32 * h), r);
          tmem_wait_ld();
          if (h == 1 && c + 64 == C::WCOLS) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(acce_lead0 + 8u * (uint32_t)acc);
          }
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          stage_row<OT, 128, 32>(buf, (uint32_t)lane, (uint32_t)(4 * h), v);
        }
        __syncwarp();
        if (rows > 0 && col0 + c < a.k)
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

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every remote arrive and copy of the pair is done before either CTA frees anything
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<2>(tmem, C::TMEM_COLS);
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
  return launch_pdl(kern, dim3((unsigned)(2 * grid)), kGradThreads, GradCfg<BN>::SMEM, s, 0, m.pw, m.px, m.x, m.w, a);
}

template <int DT>
cudaError_t launch_dp(bool vec, const void* P, const void* dY, int T, int F, int pitch, int act, void* dp, float* part,
                      cudaStream_t s) {
  const dim3 grid((unsigned)((F + kDpCols - 1) / kDpCols), (unsigned)((T + kDpRows - 1) / kDpRows));
  const uint16_t *p = static_cast<const uint16_t*>(P), *y = static_cast<const uint16_t*>(dY);
  uint16_t* o = static_cast<uint16_t*>(dp);
  auto kern = vec ? (part ? gated_dp_kernel<DT, true, true> : gated_dp_kernel<DT, true, false>)
                  : (part ? gated_dp_kernel<DT, false, true> : gated_dp_kernel<DT, false, false>);
  return launch_pdl(kern, grid, 32 * kDpWarps, 0, s, 0, p, y, T, F, pitch, act, o, part);
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: dp, the masked dense weight, the row blocks' column sums.
struct GradWs {
  int64_t pitch, dp, wm, part, total;
  GradWs(const nm_handle* h, int64_t T) {
    const int64_t F = h->n_out / 2;
    pitch = (F + 7) / 8 * 8;
    dp = 0;
    wm = dp + align256(T * 2 * pitch * 2);
    part = wm + align256(h->n_out * h->k * 2);
    total = part + align256((T + kDpRows - 1) / kDpRows * h->n_out * 4);
  }
};

nm_status check_grad(const nm_handle* h, int64_t T) {
  nm_status st = check_handle(h);
  if (st != NM_OK) return st;
  if (!h->gated || h->mx) return fail(NM_ERR_INVALID, "nm_gated_backward needs a handle made by nm_compress_gated");
  if (h->dt == DT_I8) return fail(NM_ERR_UNSUPPORTED, "gradients are for FP16 and BF16 handles only");
  if (T < 0) return fail(NM_ERR_INVALID, "T must be >= 0 (got %lld)", (long long)T);
  if (T > (int64_t(1) << 30)) return fail(NM_ERR_UNSUPPORTED, "T above 2^30");
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
  const int row_blocks = (int)((T + kDpRows - 1) / kDpRows);
  if (row_blocks > 65535) return fail(NM_ERR_UNSUPPORTED, "T above %d", 65535 * kDpRows);

  cudaError_t e = cudaSuccess;
  if (dX && (e = launch_decompress(h, base + lay.wm, s)) != cudaSuccess) return cuda_fail(e, "unpack the weight");
  const bool vec = F % 8 == 0;  // every row starts on 16 bytes
  e = h->dt == DT_F16 ? launch_dp<DT_F16>(vec, P, dY, (int)T, (int)F, (int)lay.pitch, (int)act, dp, part, s)
                      : launch_dp<DT_BF16>(vec, P, dY, (int)T, (int)F, (int)lay.pitch, (int)act, dp, part, s);
  if (e != cudaSuccess) return cuda_fail(e, "launch the gradient of the output stage");

  if (dX || dW) {
    const int pairs = num_sms(h->device) / 2;
    const int bn = h->k > 128 ? 256 : 128;
    const int n_nt = (int)((h->k + bn - 1) / bn);
    GradArgs a{};
    a.F = (int)F;
    a.T = (int)T;
    a.k = (int)h->k;
    a.dW = dW;
    a.dX = dX;
    a.err = h->d_err;
    a.timeout_ns = 1000000000ull;
    a.kb_half = (int)((F + kGradKb - 1) / kGradKb);
    GradSide sw{}, sx{};
    sw.dw = 1;
    sw.n_nt = n_nt;
    sw.n_mt = (int)((F + 255) / 256);
    sw.n_kb = (int)((T + kGradKb - 1) / kGradKb);
    sw.tiles = dW ? 2 * sw.n_mt * n_nt : 0;
    sx.n_nt = n_nt;
    sx.n_mt = (int)((T + 255) / 256);
    sx.n_kb = 2 * a.kb_half;
    const int64_t x_tiles = dX ? (int64_t)sx.n_mt * n_nt : 0;
    if (x_tiles > INT32_MAX / 2) return fail(NM_ERR_UNSUPPORTED, "T x k too large");
    sx.tiles = (int)x_tiles;
    const bool w_first = sw.n_kb >= sx.n_kb;
    a.side[0] = w_first ? sw : sx;
    a.side[1] = w_first ? sx : sw;
    const int64_t total = (int64_t)sw.tiles + sx.tiles;
    const int grid = (int)std::min<int64_t>(total, pairs);
    // Share out side 1 on top of side 0 so that the fullest pair has the least to
    // do: the lowest level L (in stages) at which every tile finds room.
    const int kFixed = 6;  // a tile's fill and drain, in stages
    const int64_t c0 = a.side[0].n_kb + kFixed, c1 = a.side[1].n_kb + kFixed;
    const int64_t q = a.side[0].tiles / grid;
    a.hi = a.side[0].tiles % grid;
    int64_t lo = 0, hi = 0;
    for (int64_t need = (a.side[1].tiles * c1 + a.side[0].tiles * c0) / grid;; need += c1 / 8 + 1) {
      lo = std::max<int64_t>(0, (need - q * c0) / c1);
      hi = a.hi ? std::max<int64_t>(0, (need - (q + 1) * c0) / c1) : lo;
      if (lo * (grid - a.hi) + hi * a.hi >= a.side[1].tiles) break;
    }
    a.lo_tiles = (int)lo;
    a.hi_tiles = (int)hi;

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
  if (dbias) {
    e = launch_pdl(dbias_kernel, dim3((unsigned)((h->n_out + 31) / 32)), 256, 0, s, 0, (const float*)part, (int)h->n_out,
                   row_blocks, dbias);
    if (e != cudaSuccess) return cuda_fail(e, "launch the bias gradient");
  }
  return NM_OK;
}

}  // extern "C"

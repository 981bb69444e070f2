// nm_mx.cu -- microscaled 4-bit floating point (include/nmspmm.h gives the
// format): quantisation of activations and weights, the values back, and the
// product of two quantised matrices on the block-scaled tensor core.
#include <cstdlib>
#include <new>
#include <string>

#include "nm_act.cuh"
#include "nm_api_internal.h"
#include "nm_device.cuh"
#include "nm_launch.cuh"
#include "nm_stage.cuh"

namespace nm {
namespace {

// ------------------------------------------------------------------ quantisation

enum : int { SRC_F16 = NM_FP16, SRC_BF16 = NM_BF16, SRC_F32 = NM_FP32 };
__host__ __device__ constexpr int src_bytes(int dt) { return dt == SRC_F32 ? 4 : 2; }

// 16 consecutive values as they lie in memory, and as fp32.  (Coherent loads, here and
// below: the kernel may have started while the one that writes its input was running.)
template <int DT>
struct Raw16 {
  uint4 q[src_bytes(DT)];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < src_bytes(DT); ++i) q[i] = __ldca(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < src_bytes(DT); ++i) q[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void to_f32(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < src_bytes(DT); ++i) {
      const uint32_t x[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == SRC_F32) {
          v[4 * i + j] = __uint_as_float(x[j]);
        } else if constexpr (DT == SRC_BF16) {
          v[8 * i + 2 * j] = __uint_as_float(x[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
          v[8 * i + 2 * j] = f.x;
          v[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
  }
};

// Zero all but the N largest magnitudes of every M values (ties keep the lower
// position): a value goes when N others precede it.
template <int N, int M>
__device__ __forceinline__ void prune16(float (&v)[16]) {
  if constexpr (N < M) {
#pragma unroll
    for (int g = 0; g < 16; g += M) {
      int before[M];
#pragma unroll
      for (int i = 0; i < M; ++i) before[i] = 0;
#pragma unroll
      for (int p = 0; p < M; ++p)
#pragma unroll
        for (int q = p + 1; q < M; ++q) {
          const int later = (__float_as_uint(v[g + q]) & 0x7FFFFFFFu) > (__float_as_uint(v[g + p]) & 0x7FFFFFFFu);
          before[p] += later;
          before[q] += 1 - later;
        }
#pragma unroll
      for (int p = 0; p < M; ++p)
        if (before[p] >= N) v[g + p] = 0.0f;
    }
  }
}

// Eight values to eight 4-bit codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// One block quantises one scale atom, 128 rows x 128 k: a thread takes 16
// values (half a scale block, its partner the other half) of a row per pass,
// eight threads a row, 32 rows a pass.  The 512 scale bytes of the atom are
// collected in shared memory and written as one run; atoms beyond k (the tile is
// 256 k wide) are written as zeros.  Memory bound: 5.3 us for 12608 x 768 bf16 (4.6
// TB/s), 10.0 for 12608 x 1024 fp32 (5.9); with the values converted as they were
// loaded (80 registers instead of 55, three blocks an SM) the former took 7.5.
//
// N < M: the values are pruned first.  n_ff > 0: packed row r comes from row
// gated_source_row(r, n_ff) of X, and `rows` counts packed rows.
template <int DT, int N, int M>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const uint8_t* __restrict__ X, int64_t rows, int64_t k,
                                                          int64_t ldx_bytes, int64_t n_ff, uint8_t* __restrict__ Q,
                                                          uint8_t* __restrict__ S, int64_t n_kb) {
  __shared__ __align__(16) uint8_t sc[512];
  pdl_launch_dependents();
  pdl_wait();
  const int atom = (int)(blockIdx.x % (2 * n_kb));        // 128-k atom along k
  const int64_t row0 = (int64_t)(blockIdx.x / (2 * n_kb)) * 128;
  const int64_t kk = (int64_t)atom * 128 + (threadIdx.x & 7) * 16;
  const int sub = threadIdx.x >> 3;
  constexpr int PASSES = 4;
  Raw16<DT> raw[PASSES];  // every pass's loads are in flight before the first is used
  bool live[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = row0 + i * 32 + sub;
    const int64_t src = r < rows ? (n_ff ? gated_source_row(r, n_ff) : r) : -1;
    live[i] = r < rows && kk < k;
    if (src >= 0 && kk < k)
      raw[i].load(X + src * ldx_bytes + kk * src_bytes(DT));
    else
      raw[i].zero();
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    float v[16];
    raw[i].to_f32(v);
    prune16<N, M>(v);
    uint32_t top = 0;  // the largest magnitude, as bits: infinities and NaN compare above all finite values
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const uint32_t eb = top >> 23;  // exponent field: floor(log2) + 127 (0 for subnormals, far below the limit)
    const bool bad = eb == 255u;
    const uint32_t byte = bad ? 255u : (eb > 2u ? eb - 2u : 0u);
    const float inv = bad ? 0.0f : __uint_as_float((254u - byte) << 23);  // 2^-(byte - 127), exact
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = bad ? 0.0f : __fmul_rn(v[j], inv);
    if (live[i]) {
      const uint2 q = make_uint2(e2m1x8(v), e2m1x8(v + 8));
      *reinterpret_cast<uint2*>(Q + (row0 + i * 32 + sub) * (k >> 1) + (kk >> 1)) = q;
    }
    if ((threadIdx.x & 1) == 0) sc[sub * 16 + i * 4 + ((threadIdx.x & 7) >> 1)] = live[i] ? (uint8_t)byte : 0;
  }
  __syncthreads();
  if (threadIdx.x < 32)
    reinterpret_cast<uint4*>(S + ((row0 >> 7) * n_kb + (atom >> 1)) * 1024 + (atom & 1) * 512)[threadIdx.x] =
        reinterpret_cast<const uint4*>(sc)[threadIdx.x];
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Four codes (the low 16 bits of q) times their block's scale (bf16, twice), as
// bf16: exact, since bf16 holds every product (or it is infinite there and in fp32).
// The codes are the selectors of byte permutes: two look up the bytes of the
// magnitude, one copies 0x80 or, for a selector with its top bit set, spreads that
// byte's sign to 0xFF, whose second highest bit is then the sign.
__device__ __forceinline__ uint2 e2m1x4_scaled(uint32_t q, uint32_t scale2) {
  const uint32_t sel = q & 0x7777u;
  const uint32_t lo = prmt(0xC0800000u, 0xC0804000u, sel);  // of 0, 0.5, 1, 1.5 and of 2, 3, 4, 6
  const uint32_t hi = prmt(0x3F3F3F00u, 0x40404040u, sel) | ((prmt(0x80808080u, 0x80808080u, q) << 1) & 0x80808080u);
  uint2 h;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(h.x) : "r"(prmt(lo, hi, 0x5140u)), "r"(scale2));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(h.y) : "r"(prmt(lo, hi, 0x7362u)), "r"(scale2));
  return h;
}

// A thread writes 16 bytes at a time (4 or 8 values), neighbours side by side, so
// that a warp instruction fills whole sectors.  Block (x, y): `block_rows` rows from
// row x * block_rows, units [y * cols, (y + 1) * cols) of each (a unit is 16 bytes
// of output).  n_ff > 0: packed rows back to their place in W.  12608 x 768 bf16 takes
// 6.3 us (3.9 TB/s; 7.2 with the values looked up as fp16 and scaled in fp32), 12608 x
// 1024 fp32 12.4 (4.7 TB/s): launch and latency beside the bytes, four units a thread;
// holding four units' loads in flight by hand changed nothing.
template <int DT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ Q,
                                                            const uint8_t* __restrict__ S, int64_t rows, int64_t k,
                                                            int64_t n_ff, int64_t n_kb, int block_rows, int cols,
                                                            uint8_t* __restrict__ X) {
  constexpr int PER = 16 / src_bytes(DT);  // values of a unit
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row0 = (int64_t)blockIdx.x * block_rows;
  const int u0 = (int)blockIdx.y * cols, width = min(cols, (int)(k / PER) - u0);
  const int nrows = (int)min((int64_t)block_rows, rows - row0);
  // unit c of row dr, advanced by the block's 256 units without a division
  const int step_r = 256 / width, step_c = 256 - step_r * width;
  int dr = (int)threadIdx.x / width, c = (int)threadIdx.x - dr * width;
  const uint8_t* q0 = Q + row0 * (k >> 1) + (int64_t)u0 * (PER / 2);
#pragma unroll 4
  for (; dr < nrows; dr += step_r, c += step_c) {
    if (c >= width) {
      c -= width;
      if (++dr >= nrows) break;
    }
    const int64_t r = row0 + dr;
    const int kk = (u0 + c) * PER;
    const int64_t dst = n_ff ? gated_source_row(r, n_ff) : r;
    if (dst < 0) continue;
    const uint8_t* qp = q0 + (int64_t)dr * (k >> 1) + c * (PER / 2);
    const uint32_t q = PER == 4 ? (uint32_t)__ldca(reinterpret_cast<const unsigned short*>(qp))
                                : __ldca(reinterpret_cast<const unsigned int*>(qp));
    const uint32_t byte = __ldca(S + mx_scale_offset(r, kk >> 5, n_kb));
    // 2^(byte - 127): a subnormal for byte 0, NaN for byte 255
    const uint32_t scale = byte == 0 ? 0x0040u : byte == 255u ? 0x7FC0u : byte << 7;
    const uint32_t scale2 = scale * 0x10001u;
    const uint2 h0 = e2m1x4_scaled(q, scale2);
    uint4 o;
    if constexpr (DT == SRC_F32) {
      o = make_uint4(h0.x << 16, h0.x & 0xFFFF0000u, h0.y << 16, h0.y & 0xFFFF0000u);
    } else {
      const uint2 h1 = e2m1x4_scaled(q >> 16, scale2);
      o = make_uint4(h0.x, h0.y, h1.x, h1.y);
      if constexpr (DT == SRC_F16) {
        uint32_t* w = &o.x;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack_pair<OUT_F16>(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      }
    }
    *reinterpret_cast<uint4*>(X + (dst * k + kk) * src_bytes(DT)) = o;
  }
}

template <int DT, int N, int M>
cudaError_t launch_quantize_t(const void* X, int64_t rows, int64_t k, int64_t ldx, int64_t n_ff, uint8_t* Q,
                              uint8_t* S, cudaStream_t s) {
  const int64_t n_kb = (k + 255) / 256, blocks = (rows + 127) / 128 * 2 * n_kb;
  return launch_pdl(mx_quantize_kernel<DT, N, M>, dim3((unsigned)blocks), 256, 0, s, 0,
                    static_cast<const uint8_t*>(X), rows, k, ldx * (int64_t)src_bytes(DT), n_ff, Q, S, n_kb);
}

template <int DT>
cudaError_t launch_quantize(int N, int M, const void* X, int64_t rows, int64_t k, int64_t ldx, int64_t n_ff,
                            uint8_t* Q, uint8_t* S, cudaStream_t s) {
  if (N == M) return launch_quantize_t<DT, 4, 4>(X, rows, k, ldx, n_ff, Q, S, s);
  switch (N * 16 + M) {
    case 1 * 16 + 4: return launch_quantize_t<DT, 1, 4>(X, rows, k, ldx, n_ff, Q, S, s);
    case 2 * 16 + 4: return launch_quantize_t<DT, 2, 4>(X, rows, k, ldx, n_ff, Q, S, s);
    case 2 * 16 + 8: return launch_quantize_t<DT, 2, 8>(X, rows, k, ldx, n_ff, Q, S, s);
    case 4 * 16 + 8: return launch_quantize_t<DT, 4, 8>(X, rows, k, ldx, n_ff, Q, S, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_quantize_dt(int dt, int N, int M, const void* X, int64_t rows, int64_t k, int64_t ldx,
                               int64_t n_ff, uint8_t* Q, uint8_t* S, cudaStream_t s) {
  switch (dt) {
    case SRC_F16: return launch_quantize<SRC_F16>(N, M, X, rows, k, ldx, n_ff, Q, S, s);
    case SRC_BF16: return launch_quantize<SRC_BF16>(N, M, X, rows, k, ldx, n_ff, Q, S, s);
    case SRC_F32: return launch_quantize<SRC_F32>(N, M, X, rows, k, ldx, n_ff, Q, S, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int DT>
cudaError_t launch_dequantize(const uint8_t* Q, const uint8_t* S, int64_t rows, int64_t k, int64_t n_ff, void* X,
                              int sms, cudaStream_t s) {
  const int64_t units = k * src_bytes(DT) / 16;  // of a row
  const int cols = (int)(units < 2048 ? units : 2048);
  // as many blocks as are resident at once (8 an SM), of 256 units at least
  const int64_t chunks = (units + cols - 1) / cols, want = (rows * chunks + 8 * sms - 1) / (8 * sms);
  const int block_rows = (int)(want * cols > 256 ? want : (256 + cols - 1) / cols);
  const dim3 grid((unsigned)((rows + block_rows - 1) / block_rows), (unsigned)((units + cols - 1) / cols));
  return launch_pdl(mx_dequantize_kernel<DT>, grid, 256, 0, s, 0, Q, S, rows, k, n_ff, (k + 255) / 256, block_rows, cols,
                    static_cast<uint8_t*>(X));
}

// ------------------------------------------------------------------ product
//
// Two CTAs on two SMs compute a tile of 256 tokens x BN channels with
// tcgen05.mma.cta_group::2.kind::mxf4 (block scales of 32 k): A is the quantised
// activation (each CTA's 128 token rows), B the quantised weight (each CTA BN/2
// of the tile's channel rows).  A k-block is 256 k: 128 bytes of codes per row, in
// the same K-major 128-byte-swizzled operand layout as every other type, plus two
// 512-byte scale atoms per 128 rows, which tcgen05.cp spreads into tensor memory
// (lane l, column q: the four scale bytes of row 32 q + l).  Each CTA needs the
// scales of its own token rows and of all BN channels.
//
// Tokens are the accumulator's lanes, so a thread holds consecutive channels of
// one token: scale, bias and activation need no exchange between threads, the
// two halves of a gated pair (16 gate channels beside their 16 up channels) meet
// in one thread, and rows leave through a staged tile as whole lines.
//
// What bounds it.  A stage (256 k of a 192-channel tile) takes 0.22 us, 430 cycles
// against 384 of MMA; a 64-channel tile's takes 0.21, the issuing lane's own
// instructions.  12608 x 1024 -> 4096: 35 us with bf16 output (the output stage and the
// mainloop share the SM's shared memory and issue slots), 45 with bias and GELU (issue
// 58 %, XU 28 %, MMA 25 %: the warps of a tile run through wait, arithmetic and stores
// together; halves of them on alternate tiles took 47 against 46 then).  At k = 8192 it
// runs at 5.6 PFLOP/s.  Narrower tiles (128, 64 channels: 47 and 58 us on that case)
// serve fewer tokens: 197 x 768 -> 2 x 2048 takes 5.0 us with 192, 4.5 and 4.6 with them.
constexpr int kMxKb = 256;
constexpr int kMxSmemBudget = 227 * 1024 - 1024 - 512;  // 1 KB of alignment slack, barriers

template <int BN, bool GATED>
struct MxCfg {
  static constexpr int HB = BN / 2;                            // channel rows each CTA loads
  static constexpr int ATOMS = BN > 128 ? 2 : 1;               // 128-channel scale tiles that cover BN channels
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = HB * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES + 1024 + ATOMS * 1024;
  // Accumulator columns per epilogue warp: 32, or 64 for gated tiles (32 outputs,
  // a 64-byte run of a 16-bit row).  12608 x 1024 -> 4096 with bias and GELU takes
  // 45.9 us with 32 columns a warp (24 warps of 72 registers) and 47.8 with 64; gated
  // 12608 x 768 -> 2 x 2048 33.1 with 32 and 27.3 with 64.
  static constexpr int WCOLS = GATED && BN > 64 ? 64 : 32;
  static constexpr int EPW = BN / WCOLS;                       // epilogue warps per lane quarter
  static constexpr int EPI_WARPS = 4 * EPW;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int EPI_BUF = 2048;                         // per warp: 32 staged rows of 64 bytes
  static constexpr int EPI_BYTES = EPI_WARPS * EPI_BUF;
  static constexpr int VEC_BYTES = EPI_WARPS * 2 * WCOLS * 4;  // (static) scale and bias of each warp's columns
  static constexpr int STAGES_FIT = (kMxSmemBudget - EPI_BYTES - VEC_BYTES) / STAGE;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr int SMEM = STAGES * STAGE + EPI_BYTES + 1024;
  static constexpr int SF_COLS = 8 + 8 * ATOMS;                // scale columns of one stage
  static constexpr int COLS_NEEDED = 2 * BN + 2 * SF_COLS;
  static constexpr int TMEM_COLS = COLS_NEEDED <= 256 ? 256 : 512;
  static_assert(STAGE % 1024 == 0 && B_BYTES % 1024 == 0, "stages keep 1024-byte alignment");
  static_assert(STAGES >= 3 && COLS_NEEDED <= 512 && WCOLS % 32 == 0, "tile fits");
  // a tile starts at a multiple of BN: 64 rows into a scale tile at most
  static_assert(128 % BN == 0 || (BN - 64) % 128 == 0, "scale tiles cover the channels");
};

struct MxArgs {
  void* Y;
  const float* scale;
  const float* bias;
  int* err;
  int T, n_y, n_acc, n_ff;   // tokens; output channels; accumulator channels; gated: n_ff, else 0
  int k, n_kb, n_tb, n_rb;   // k, 256-k blocks, 128-row scale tiles of X and of the weight
  int n_nt, units;
  int out_ty, act;
  int vec;                   // rows of Y start on 16 bytes
  int a_rows;                // token rows of a copy of X
  unsigned long long timeout_ns;
};

// A: e2m1, B: e2m1, fp32 accumulation, E8M0 scales; the data ids (bits 4-5 and
// 29-30) choose bytes 0-1 or 2-3 of each row's four scale bytes.
template <int BN>
__host__ __device__ constexpr uint32_t mx_idesc(uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((256u >> 4) << 24) |
         (sf_id << 29);
}

// A pair's tiles, u_step apart, without a division at each (an epilogue warp of 32
// columns runs some 500 instructions a tile).
struct MxWalk {
  int u, nt, mt;
  int n_nt, du, dn, dm;
  __device__ __forceinline__ MxWalk(int first, int step, int n)
      : u(first), nt(first % n), mt(first / n), n_nt(n), du(step), dn(step % n), dm(step / n) {}
  __device__ __forceinline__ int next_nt() const { return nt + dn >= n_nt ? nt + dn - n_nt : nt + dn; }
  __device__ __forceinline__ void next() {
    u += du;
    nt += dn;
    mt += dm;
    if (nt >= n_nt) {
      nt -= n_nt;
      ++mt;
    }
  }
};

// Scale and bias of a warp's accumulator columns, one column of every 32 per lane.
template <int WCOLS, bool GATED>
struct MxVectors {
  float s[WCOLS / 32], b[WCOLS / 32];
  __device__ __forceinline__ void fetch(const MxArgs& a, int col0, int lane) {
#pragma unroll
    for (int c = 0; c < WCOLS / 32; ++c) {
      const int ch = col0 + 32 * c + lane;
      int src = ch;
      bool in = ch < a.n_acc;
      if constexpr (GATED) {
        const int f = (ch >> 5) * 16 + (ch & 15);
        in = f < a.n_ff;
        src = (ch & 16) ? a.n_ff + f : f;
      }
      s[c] = a.scale && in ? ld_coherent(a.scale + src) : 0.0f;
      b[c] = a.bias && in ? ld_coherent(a.bias + src) : 0.0f;
    }
  }
  // Into shared memory, where every lane reads them all.
  __device__ __forceinline__ void publish(const MxArgs& a, float* vs, float* vb, int lane) const {
    if (!a.scale && !a.bias) return;
    __syncwarp();  // the previous tile's reads are done
#pragma unroll
    for (int c = 0; c < WCOLS / 32; ++c) {
      vs[32 * c + lane] = s[c];
      vb[32 * c + lane] = b[c];
    }
    __syncwarp();
  }
};

// The output stage of one epilogue warp: WCOLS accumulator columns of its 32
// tokens, all in registers (v).  32 columns at a time: scale, bias, activation
// (and gate), then staged rows of 64 bytes.
template <int OT, int WCOLS, bool GATED>
__device__ __forceinline__ void mx_epilogue(const MxArgs& a, float (&v)[WCOLS], uint8_t* buf, const float* vs,
                                            const float* vb, int row0, int col0, int lane) {
  constexpr int ES = stage_elem_bytes(OT);
  constexpr int NV = GATED ? 16 : 32;            // outputs of one step of 32 columns
  constexpr int PER = 64 / ES;                   // outputs of a staged row
  constexpr int TOTAL = WCOLS / 32 * NV;         // outputs of this warp per token
  const int rows = min(32, a.T - row0);
  if (a.scale) {
#pragma unroll
    for (int j = 0; j < WCOLS; j += 4) {
      const float4 s4 = *reinterpret_cast<const float4*>(vs + j);
      upk2(mul2(pk2(v[j], v[j + 1]), pk2(s4.x, s4.y)), v[j], v[j + 1]);
      upk2(mul2(pk2(v[j + 2], v[j + 3]), pk2(s4.z, s4.w)), v[j + 2], v[j + 3]);
    }
  }
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < WCOLS; j += 4) {
      const float4 b4 = *reinterpret_cast<const float4*>(vb + j);
      upk2(add2(pk2(v[j], v[j + 1]), pk2(b4.x, b4.y)), v[j], v[j + 1]);
      upk2(add2(pk2(v[j + 2], v[j + 3]), pk2(b4.z, b4.w)), v[j + 2], v[j + 3]);
    }
  }
#pragma unroll
  for (int c = 0; c < WCOLS / 32; ++c) {
    act_run<NV>(v + 32 * c, a.act);
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[16 * c + j] = __fmul_rn(v[32 * c + j], v[32 * c + 16 + j]);
    }
  }
  // outputs v[0 .. TOTAL)
#pragma unroll
  for (int o = 0; o < TOTAL; o += PER) {
    constexpr int N = TOTAL < PER ? TOTAL : PER;
    if (o > 0) __syncwarp();
    stage_row<OT, 64, N>(buf, (uint32_t)lane, 0, v + o);
    __syncwarp();
    const int ycol = (GATED ? col0 / 2 : col0) + o;
    if (rows > 0 && ycol < a.n_y)
      stage_flush<64, ES>(buf, static_cast<uint8_t*>(a.Y) + ((int64_t)row0 * a.n_y + ycol) * ES, (int64_t)a.n_y * ES, rows,
                      min(N, a.n_y - ycol) * ES, a.vec != 0, lane);
  }
  __syncwarp();
}

template <int BN, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MxCfg<BN, GATED>::THREADS, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const MxArgs a) {
  using C = MxCfg<BN, GATED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(16) float vec_sh[C::EPI_WARPS][2][C::WCOLS];
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
      mbar_init(&acce_bar[i], 2 * C::EPI_WARPS);  // both CTAs' epilogue warps
    }
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    prefetch_tensormap(&tmSA);
    prefetch_tensormap(&tmSB);
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
  const int u_first = (int)cluster_id_x(), u_step = (int)nclusters_x();

  auto give_up = [&](int code) {
    abort_sh = 1;
    if (a.err) atomicExch(a.err, code);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    // One lane runs this loop, and one the next: with whole warps around the issuing
    // lane, their instructions made a stage take 0.25 us whatever the tile's width
    // (0.21 so; three stages in the ring were as good as eight).
    uint32_t issued = 0;
    if (elect_one()) {
      const uint32_t stage_tx = 2u * (uint32_t)(C::STAGE - C::A_BYTES + a.a_rows * 128);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint8_t* st = smem;
      uint32_t fb = full_lead0;
      for (MxWalk w(u_first, u_step, a.n_nt); ok && w.u < a.units; w.next()) {
        const int arow = w.mt * 256 + (int)rank * 128;
        const int brow = w.nt * BN + (int)rank * C::HB;
        const int btile = (w.nt * BN) >> 7;
        // the last tile's second half may lie behind the last scale tile: any
        // tile's scales do for rows that are not stored
        const int srow = min(2 * w.mt + (int)rank, a.n_tb - 1) * a.n_kb * 8;
        int brow8[C::ATOMS];
#pragma unroll
        for (int i = 0; i < C::ATOMS; ++i) brow8[i] = min(btile + i, a.n_rb - 1) * a.n_kb * 8;
        for (int kb = 0; kb < a.n_kb; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_sh, tmo)) {
            give_up(1);
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], stage_tx);
          tma_load_2d_pair(st, &tmA, fb, kb * 128, arow);
          tma_load_2d_pair(st + C::A_BYTES, &tmB, fb, kb * 128, brow);
          tma_load_2d_pair(st + C::A_BYTES + C::B_BYTES, &tmSA, fb, 0, srow + kb * 8);
#pragma unroll
          for (int i = 0; i < C::ATOMS; ++i)
            tma_load_2d_pair(st + C::A_BYTES + C::B_BYTES + 1024 + i * 1024, &tmSB, fb, 0, brow8[i] + kb * 8);
          ++issued;
          st += C::STAGE;
          fb += 8;
          if (++stage == C::STAGES) {
            stage = 0;
            st = smem;
            fb = full_lead0;
            phase ^= 1u;
          }
        }
      }
      if (leader)  // drain: both CTAs' copies have landed (the peer is held by the cluster barrier below)
        for (uint32_t i = issued > (uint32_t)C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
          mbar_wait(&full_bar[i % C::STAGES], (i / C::STAGES) & 1u, &abort_sh, tmo);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (leader) {
      if (elect_one()) {
        int stage = 0, acc = 0, slot = 0;
        uint32_t phase = 0, acc_phase = 0, off = 0;  // off: the stage's offset in the descriptors' address fields
        const uint32_t base = smem_u32(smem);
        const uint64_t ad_base = sdesc_sw128(base), bd_base = sdesc_sw128(base + C::A_BYTES);
        const uint64_t sa_base = sdesc_rows16(base + C::A_BYTES + C::B_BYTES);
        bool ok = true;
        for (MxWalk w(u_first, u_step, a.n_nt); ok && w.u < a.units; w.next()) {
          const uint32_t sfb_off = (uint32_t)(((w.nt * BN) & 127) >> 5);  // the tile's first channel within its scale tile
          if (!mbar_wait(&acce_bar[acc], acc_phase ^ 1u, &abort_sh, tmo)) {
            give_up(2);
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
          for (int kb = 0; kb < a.n_kb; ++kb) {
            if (!mbar_wait(&full_bar[stage], phase, &abort_sh, tmo)) {
              give_up(3);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad0 = ad_base + off, bd0 = bd_base + off, sa0 = sa_base + off;
            const uint32_t sfa = tmem + (uint32_t)(2 * BN + slot * C::SF_COLS), sfb = sfa + 8;
            const int mmas = min(4, (a.k - kb * kMxKb + 63) >> 6);  // k beyond the matrix is skipped in steps of 64
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tc_cp_32x128b_x4_pair(sfa + 4 * h, sa0 + 32u * h);
#pragma unroll
              for (int i = 0; i < C::ATOMS; ++i)
                tc_cp_32x128b_x4_pair(sfb + 4 * C::ATOMS * h + 4 * i, sa0 + 64u + 64u * i + 32u * h);
            }
            if (mmas == 4) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_mxf4_pair(d_tmem, ad0 + 2u * j, bd0 + 2u * j, (j & 1) ? mx_idesc<BN>(2) : mx_idesc<BN>(0),
                                 sfa + 4 * (j >> 1), sfb + 4 * C::ATOMS * (j >> 1) + sfb_off,
                                 (kb > 0 || j > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int j = 0; j < 3; ++j)
                if (j < mmas)
                  tc_mma_mxf4_pair(d_tmem, ad0 + 2u * j, bd0 + 2u * j, (j & 1) ? mx_idesc<BN>(2) : mx_idesc<BN>(0),
                                   sfa + 4 * (j >> 1), sfb + 4 * C::ATOMS * (j >> 1) + sfb_off,
                                   (kb > 0 || j > 0) ? 1u : 0u);
            }
            tc_commit_pair(&empty_bar[stage], (uint16_t)3);
            slot ^= 1;
            off += C::STAGE >> 4;
            if (++stage == C::STAGES) {
              stage = 0;
              off = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit_pair(&accf_bar[acc], (uint16_t)3);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        tc_commit_pair(&drain_bar, (uint16_t)3);
      }
      __syncwarp();
    }
    mbar_wait_warp(&drain_bar, 0, &abort_sh, tmo);  // every MMA of this pair has completed
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int ew = warp - 2, lq = warp & 3, part = ew >> 2;
    uint8_t* buf = smem + (size_t)C::STAGES * C::STAGE + (size_t)ew * C::EPI_BUF;
    float* vs = vec_sh[ew][0];
    float* vb = vec_sh[ew][1];
    int acc = 0;
    uint32_t acc_phase = 0;
    MxVectors<C::WCOLS, GATED> vec;  // of the next tile: fetched a tile ahead
    MxWalk w(u_first, u_step, a.n_nt);
    vec.fetch(a, w.nt * BN + part * C::WCOLS, lane);
    for (; w.u < a.units; w.next()) {
      const int row0 = w.mt * 256 + (int)rank * 128 + lq * 32;
      const int col0 = w.nt * BN + part * C::WCOLS;
      vec.publish(a, vs, vb, lane);
      vec.fetch(a, w.next_nt() * BN + part * C::WCOLS, lane);
      if (!mbar_wait_warp(&accf_bar[acc], acc_phase, &abort_sh, tmo)) {
        if (lane == 0) give_up(4);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(lq * 32) << 16) + (uint32_t)(acc * BN + part * C::WCOLS);
      float v[C::WCOLS];
      __syncwarp();
#pragma unroll
      for (int c = 0; c < C::WCOLS; c += 32) tmem_ld32(taddr + (uint32_t)c, *reinterpret_cast<uint32_t(*)[32]>(v + c));
      tmem_wait_ld();
      // all of this warp's columns are in registers: release the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(acce_lead0 + 8u * (uint32_t)acc);
      switch (a.out_ty) {
        case OUT_F16: mx_epilogue<OUT_F16, C::WCOLS, GATED>(a, v, buf, vs, vb, row0, col0, lane); break;
        case OUT_BF16: mx_epilogue<OUT_BF16, C::WCOLS, GATED>(a, v, buf, vs, vb, row0, col0, lane); break;
        default: mx_epilogue<OUT_F32, C::WCOLS, GATED>(a, v, buf, vs, vb, row0, col0, lane); break;
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

// Channel tiles of the product and the box heights of the weight's tensor maps.
constexpr int kMxTiles[3] = {192, 128, 64};

template <int BN, bool GATED>
cudaError_t launch_mx_t(const nm_handle* h, int slot, int grid, const CUtensorMap& tmA, const CUtensorMap& tmSA,
                        const MxArgs& a, cudaStream_t s) {
  using C = MxCfg<BN, GATED>;
  auto kern = mx_pair_kernel<BN, GATED>;
  static std::atomic<uint64_t> opted{0};
  cudaError_t e = smem_opt_in(kern, C::SMEM, opted);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(2 * grid)), C::THREADS, C::SMEM, s, 0, tmA, h->tm_mxq[slot], tmSA, h->tm_mxs,
                    a);
}

template <bool GATED>
cudaError_t launch_mx(const nm_handle* h, int slot, int grid, const CUtensorMap& tmA, const CUtensorMap& tmSA,
                      const MxArgs& a, cudaStream_t s) {
  switch (slot) {
    case 0: return launch_mx_t<kMxTiles[0], GATED>(h, slot, grid, tmA, tmSA, a, s);
    case 1: return launch_mx_t<kMxTiles[1], GATED>(h, slot, grid, tmA, tmSA, a, s);
    default: return launch_mx_t<kMxTiles[2], GATED>(h, slot, grid, tmA, tmSA, a, s);
  }
}

nm_status check_mx_matrix(int64_t rows, int64_t k) {
  if (rows < 0) return fail(NM_ERR_INVALID, "the number of rows must be >= 0 (got %lld)", (long long)rows);
  if (k <= 0 || k % 32 != 0)
    return fail(NM_ERR_INVALID, "k must be positive and a multiple of 32 (got %lld)", (long long)k);
  if (rows > INT32_MAX || k > (1 << 24)) return fail(NM_ERR_UNSUPPORTED, "more than 2^31-1 rows or k above 2^24");
  return NM_OK;
}

int64_t scale_bytes(int64_t rows, int64_t k) { return (rows + 127) / 128 * ((k + 255) / 256) * 1024; }

// Codes [rows][k / 2] as the K-major operand: 128 bytes x `box_rows` rows.
nm_status codes_map(CUtensorMap* m, const void* Q, int64_t rows, int64_t k, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)(k / 2), (uint64_t)rows}, strides[1] = {(uint64_t)(k / 2)};
  const uint32_t box[2] = {128, (uint32_t)box_rows};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, Q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// Scale tiles as rows of 128 bytes, eight to a tile.
nm_status scales_map(CUtensorMap* m, const void* S, int64_t bytes) {
  const uint64_t dims[2] = {128, (uint64_t)(bytes / 128)}, strides[1] = {128};
  const uint32_t box[2] = {128, 8};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, S, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

// Validates ep for a microscaled handle.
nm_status resolve_mx_epilogue(const nm_handle* h, const nm_epilogue* ep, bool gated, int* out_ty) {
  nm_out_type out = ep ? ep->out : NM_OUT_DEFAULT;
  if ((int)out < 0 || (int)out > 5) return fail(NM_ERR_INVALID, "unknown output type %d", (int)out);
  if (ep) {
    if ((int)ep->act < 0 || (int)ep->act > (int)NM_ACT_RELU)
      return fail(NM_ERR_INVALID, "unknown activation %d", (int)ep->act);
    if (!gated && ep->act > NM_ACT_GELU)
      return fail(NM_ERR_UNSUPPORTED, "activation %d is for gated products only", (int)ep->act);
    if ((ep->scale && !aligned(ep->scale, 4)) || (ep->bias && !aligned(ep->bias, 4)))
      return fail(NM_ERR_INVALID, "scale and bias must be 4-byte aligned");
  }
  if (out == NM_OUT_INT32 || out == NM_OUT_INT8)
    return fail(NM_ERR_UNSUPPORTED, "integer outputs need an INT8 handle");
  if (out == NM_OUT_DEFAULT)
    out = h->src_dt == NM_FP32 ? NM_OUT_FP32 : h->src_dt == NM_FP16 ? NM_OUT_FP16 : NM_OUT_BF16;
  *out_ty = out == NM_OUT_FP32 ? OUT_F32 : out == NM_OUT_FP16 ? OUT_F16 : OUT_BF16;
  return NM_OK;
}

nm_status mx_product(const nm_handle* h, const void* Q, const void* S, int64_t T, void* Y, const nm_epilogue* ep,
                     void* stream, bool gated) {
  clear_error();
  nm_status st = check_handle(h);
  if (st != NM_OK) return st;
  if (!h->mx) return fail(NM_ERR_INVALID, "the handle was not made by nm_compress_mx");
  if (gated != (h->gated != 0))
    return fail(NM_ERR_INVALID, gated ? "the handle is not gated: its product is nm_spmm_mx"
                                      : "the handle is gated: its product is nm_spmm_mx_gated");
  MxArgs a{};
  if ((st = resolve_mx_epilogue(h, ep, gated, &a.out_ty)) != NM_OK) return st;
  if (T < 0) return fail(NM_ERR_INVALID, "T must be >= 0 (got %lld)", (long long)T);
  if (T == 0) return NM_OK;
  if (T > INT32_MAX) return fail(NM_ERR_UNSUPPORTED, "T above 2^31-1");
  if (!Q || !S || !Y) return fail(NM_ERR_INVALID, "null Q, S or Y");
  if (!aligned(Q, 16) || !aligned(S, 16) || !aligned(Y, 16))
    return fail(NM_ERR_INVALID, "Q, S and Y must be 16-byte aligned");
  const int64_t n_y = gated ? h->n_out / 2 : h->n_out;
  const int es = a.out_ty == OUT_F32 ? 4 : 2;
  const size_t ybytes = (size_t)T * n_y * es, sbytes = (size_t)scale_bytes(T, h->k);
  if (overlaps(Y, ybytes, Q, (size_t)T * (h->k / 2)) || overlaps(Y, ybytes, S, sbytes))
    return fail(NM_ERR_INVALID, "Y overlaps Q or S");

  a.Y = Y;
  a.scale = ep ? ep->scale : nullptr;
  a.bias = ep ? ep->bias : nullptr;
  a.act = ep ? (int)ep->act : (gated ? ACT_SILU : ACT_NONE);
  a.err = h->d_err;
  a.T = (int)T;
  a.n_y = (int)n_y;
  a.n_acc = (int)h->mx_rows;
  a.n_ff = gated ? (int)n_y : 0;
  a.k = (int)h->k;
  a.n_kb = (int)((h->k + kMxKb - 1) / kMxKb);
  a.n_tb = (int)((T + 127) / 128);
  a.n_rb = (int)((h->mx_rows + 127) / 128);
  a.timeout_ns = 1000000000ull;
  // Channel tile: the least rounds x (tile + fixed part) over the resident pairs.
  const int pairs = num_sms(h->device) / 2;
  const int64_t n_mt = (T + 255) / 256;
  const char* forced = getenv("NMSPMM_FORCE_MX_BN");  // tests and sweeps
  const int forced_bn = forced && *forced ? atoi(forced) : 0;
  int slot = 0;
  double best = 1e300;
  for (int i = 0; i < 3; ++i) {
    if (forced_bn && kMxTiles[i] != forced_bn) continue;
    const int64_t units = n_mt * ((h->mx_rows + kMxTiles[i] - 1) / kMxTiles[i]);
    const double cost = (double)((units + pairs - 1) / pairs) * (kMxTiles[i] + 64);
    if (cost < best) {
      best = cost;
      slot = i;
    }
  }
  if (best == 1e300) return fail(NM_ERR_INVALID, "NMSPMM_FORCE_MX_BN must be 64, 128 or 192");
  const int bn = kMxTiles[slot];
  a.n_nt = (int)((h->mx_rows + bn - 1) / bn);
  const int64_t units = n_mt * a.n_nt;
  if (units > INT32_MAX) return fail(NM_ERR_UNSUPPORTED, "T x n_out too large");
  a.units = (int)units;

  CUtensorMap tmA, tmSA;
  // Fewer than 128 tokens: the copies bring in those rows alone (whole swizzle groups
  // of 8).  The operand's other rows hold what the stage held before; they reach
  // only accumulator rows that are not stored.
  a.a_rows = T < 128 ? (int)((T + 7) / 8 * 8) : 128;
  if ((st = codes_map(&tmA, Q, T, h->k, a.a_rows)) != NM_OK) return st;
  if ((st = scales_map(&tmSA, S, (int64_t)sbytes)) != NM_OK) return st;
  a.vec = (n_y * es) % 16 == 0 ? 1 : 0;
  const int grid = (int)(units < pairs ? units : pairs);
  cudaError_t e = gated ? launch_mx<true>(h, slot, grid, tmA, tmSA, a, (cudaStream_t)stream)
                        : launch_mx<false>(h, slot, grid, tmA, tmSA, a, (cudaStream_t)stream);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "launch the microscaled product");
}

}  // namespace

cudaError_t launch_mx_pack(const nm_handle* h, const void* W, cudaStream_t s) {
  return launch_quantize_dt(h->src_dt, h->N, h->M, W, h->mx_rows, h->k, h->k, h->gated ? h->n_out / 2 : 0, h->d_mxq,
                            h->d_mxs, s);
}

cudaError_t launch_mx_unpack(const nm_handle* h, void* W, cudaStream_t s) {
  return launch_dequantize<SRC_BF16>(h->d_mxq, h->d_mxs, h->mx_rows, h->k, h->gated ? h->n_out / 2 : 0, W,
                                     num_sms(h->device), s);
}

}  // namespace nm

using namespace nm;

extern "C" {

nm_status nm_mx_scale_bytes(int64_t rows, int64_t k, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(NM_ERR_INVALID, "null output");
  nm_status st = check_mx_matrix(rows, k);
  if (st != NM_OK) return st;
  *bytes = (size_t)scale_bytes(rows, k);
  return NM_OK;
}

nm_status nm_mx_quantize(const void* X, int64_t T, int64_t k, int64_t ldx, nm_dtype dt, void* Q, void* S,
                         void* stream) {
  clear_error();
  if (dt != NM_FP32 && dt != NM_FP16 && dt != NM_BF16)
    return fail(NM_ERR_INVALID, "nm_mx_quantize takes FP32, FP16 or BF16 (got dtype %d)", (int)dt);
  nm_status st = check_mx_matrix(T, k);
  if (st != NM_OK) return st;
  const int es = dt == NM_FP32 ? 4 : 2;
  if (ldx < k) return fail(NM_ERR_INVALID, "ldx=%lld is below k=%lld", (long long)ldx, (long long)k);
  if ((ldx * es) % 16 != 0)
    return fail(NM_ERR_INVALID, "ldx * sizeof(dtype) must be a multiple of 16 bytes (ldx=%lld)", (long long)ldx);
  if (T == 0) return NM_OK;
  if (!X || !Q || !S) return fail(NM_ERR_INVALID, "null X, Q or S");
  if (!aligned(X, 16) || !aligned(Q, 16) || !aligned(S, 16))
    return fail(NM_ERR_INVALID, "X, Q and S must be 16-byte aligned");
  const size_t xbytes = ((size_t)(T - 1) * ldx + k) * es, qbytes = (size_t)T * (k / 2);
  const size_t sbytes = (size_t)scale_bytes(T, k);
  if (overlaps(X, xbytes, Q, qbytes) || overlaps(X, xbytes, S, sbytes) || overlaps(Q, qbytes, S, sbytes))
    return fail(NM_ERR_INVALID, "X, Q and S overlap");
  if ((T + 127) / 128 * 2 * ((k + 255) / 256) > INT32_MAX) return fail(NM_ERR_UNSUPPORTED, "T x k too large");
  cudaError_t e = launch_quantize_dt((int)dt, 4, 4, X, T, k, ldx, 0, static_cast<uint8_t*>(Q),
                                     static_cast<uint8_t*>(S), (cudaStream_t)stream);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "launch the quantisation");
}

nm_status nm_mx_dequantize(const void* Q, const void* S, int64_t T, int64_t k, nm_dtype dt, void* X, void* stream) {
  clear_error();
  if (dt != NM_FP32 && dt != NM_FP16 && dt != NM_BF16)
    return fail(NM_ERR_INVALID, "nm_mx_dequantize gives FP32, FP16 or BF16 (got dtype %d)", (int)dt);
  nm_status st = check_mx_matrix(T, k);
  if (st != NM_OK) return st;
  if (T == 0) return NM_OK;
  if (!X || !Q || !S) return fail(NM_ERR_INVALID, "null Q, S or X");
  if (!aligned(X, 16) || !aligned(Q, 16) || !aligned(S, 16))
    return fail(NM_ERR_INVALID, "Q, S and X must be 16-byte aligned");
  const size_t xbytes = (size_t)T * k * (dt == NM_FP32 ? 4 : 2);
  if (overlaps(X, xbytes, Q, (size_t)T * (k / 2)) || overlaps(X, xbytes, S, (size_t)scale_bytes(T, k)))
    return fail(NM_ERR_INVALID, "X overlaps Q or S");
  const uint8_t *q = static_cast<const uint8_t*>(Q), *s = static_cast<const uint8_t*>(S);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "query the current device");
  const int sms = num_sms(dev);
  e = dt == NM_FP32   ? launch_dequantize<SRC_F32>(q, s, T, k, 0, X, sms, (cudaStream_t)stream)
      : dt == NM_FP16 ? launch_dequantize<SRC_F16>(q, s, T, k, 0, X, sms, (cudaStream_t)stream)
                      : launch_dequantize<SRC_BF16>(q, s, T, k, 0, X, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? NM_OK : cuda_fail(e, "launch the dequantisation");
}

nm_status nm_compress_mx(const void* W, int64_t n_out, int64_t k, nm_dtype dt, int N, int M, int gated, void* stream,
                         nm_handle** out) {
  clear_error();
  if (!out) return fail(NM_ERR_INVALID, "null output handle pointer");
  *out = nullptr;
  if (!W) return fail(NM_ERR_INVALID, "null W");
  if (dt != NM_FP32 && dt != NM_FP16 && dt != NM_BF16)
    return fail(NM_ERR_INVALID, "nm_compress_mx takes FP32, FP16 or BF16 (got dtype %d)", (int)dt);
  if (n_out <= 0) return fail(NM_ERR_INVALID, "n_out must be positive");
  nm_status st = check_mx_matrix(n_out, k);
  if (st != NM_OK) return st;
  if (n_out > (1 << 24)) return fail(NM_ERR_UNSUPPORTED, "n_out is limited to 2^24");
  if (gated && n_out % 2 != 0) return fail(NM_ERR_INVALID, "a gated weight has an even number of rows (got %lld)",
                                           (long long)n_out);
  if (M <= 0 || N <= 0 || N > M) return fail(NM_ERR_INVALID, "bad N:M %d:%d", N, M);
  bool sp24 = false;
  if (!pattern_supported(N, M, &sp24)) return fail(NM_ERR_UNSUPPORTED, "N:M %d:%d is not supported", N, M);
  if (!aligned(W, 16)) return fail(NM_ERR_INVALID, "W must be 16-byte aligned");
  if ((n_out + 159) / 128 * 2 * ((k + 255) / 256) > INT32_MAX) return fail(NM_ERR_UNSUPPORTED, "n_out x k too large");

  nm_handle* h = new (std::nothrow) nm_handle();
  if (!h) return fail(NM_ERR_OOM, "host allocation failed");
  cudaGetDevice(&h->device);
  h->n_out = n_out;
  h->k = k;
  h->N = N;
  h->M = M;
  h->dt = NM_MXFP4;
  h->mx = 1;
  h->gated = gated ? 1 : 0;
  h->src_dt = (int)dt;
  h->mx_rows = gated ? gated_packed_rows(n_out / 2) : n_out;
  h->mxs_bytes = (size_t)scale_bytes(h->mx_rows, k);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  Arena arena;
  const size_t at_q = arena.add((size_t)h->mx_rows * (k / 2)), at_s = arena.add(h->mxs_bytes), at_err = arena.add(sizeof(int));
  if ((e = arena.allocate(h)) == cudaSuccess) {
    h->d_mxq = arena.base + at_q;
    h->d_mxs = arena.base + at_s;
    h->d_err = reinterpret_cast<int*>(arena.base + at_err);
  }
  if (e != cudaSuccess) st = cuda_fail(e, "allocate the quantised weight");
  else if ((e = cudaMemsetAsync(h->d_err, 0, sizeof(int), s)) != cudaSuccess) st = cuda_fail(e, "clear error word");
  else if ((e = launch_mx_pack(h, W, s)) != cudaSuccess) st = cuda_fail(e, "launch the quantisation");
  for (int i = 0; i < 3 && st == NM_OK; ++i) st = codes_map(&h->tm_mxq[i], h->d_mxq, h->mx_rows, k, kMxTiles[i] / 2);
  if (st == NM_OK) st = scales_map(&h->tm_mxs, h->d_mxs, (int64_t)h->mxs_bytes);
  if (st != NM_OK) {
    const std::string msg = nm_last_error();
    nm_destroy(h);
    fail(st, "%s", msg.c_str());
    return st;
  }
  *out = h;
  return NM_OK;
}

nm_status nm_spmm_mx(const nm_handle* h, const void* Q, const void* S, int64_t T, void* Y, const nm_epilogue* ep,
                     void* stream) {
  return mx_product(h, Q, S, T, Y, ep, stream, false);
}

nm_status nm_spmm_mx_gated(const nm_handle* h, const void* Q, const void* S, int64_t T, void* Y,
                           const nm_epilogue* ep, void* stream) {
  return mx_product(h, Q, S, T, Y, ep, stream, true);
}

}  // extern "C"

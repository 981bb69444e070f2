// nm_stage.cuh -- output staging of the kernels whose accumulator lanes are
// output rows: each thread of a warp holds a run of one row's columns.  The warp's
// 32 rows go through a small swizzled buffer in shared memory and leave as
// 16-byte stores along the rows, so that a warp instruction writes whole 128-byte
// lines.  (Measured on the 4-bit product, 12608 x 4096 bf16 output: the same
// tile leaving by tensor stores of 64-byte rows took 5-6 cycles a row and bound
// the kernel at 34 us whatever its k.)
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nm_device.cuh"

namespace nm {

__host__ __device__ constexpr int stage_elem_bytes(int ot) { return ot == OUT_F32 ? 4 : 2; }

// Byte offset of 16-byte piece c of row `row` in a staged tile with rows of ROWB
// bytes: pieces are permuted within a row so that neither a thread's writes of its
// own row nor the reads along the rows meet in a bank.
template <int ROWB>
__device__ __forceinline__ uint32_t stage_off(uint32_t row, uint32_t c) {
  static_assert(ROWB == 128 || ROWB == 64, "staged row widths");
  const uint32_t x = ROWB == 128 ? (row & 7u) : ((row >> 1) & 3u);
  return row * (uint32_t)ROWB + ((c ^ x) << 4);
}

template <int OT>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (OT == OUT_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// NV values of this thread's row into the staged tile, from 16-byte piece c0 on.
template <int OT, int ROWB, int NV>
__device__ __forceinline__ void stage_row(uint8_t* buf, uint32_t row, uint32_t c0, const float* v) {
#pragma unroll
  for (int c = 0; c < NV * stage_elem_bytes(OT) / 16; ++c) {
    uint4 q;
    if constexpr (OT == OUT_F32) {
      q = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                     __float_as_uint(v[4 * c + 3]));
    } else {
      q = make_uint4(pack_pair<OT>(v[8 * c], v[8 * c + 1]), pack_pair<OT>(v[8 * c + 2], v[8 * c + 3]),
                     pack_pair<OT>(v[8 * c + 4], v[8 * c + 5]), pack_pair<OT>(v[8 * c + 6], v[8 * c + 7]));
    }
    *reinterpret_cast<uint4*>(buf + stage_off<ROWB>(row, c0 + (uint32_t)c)) = q;
  }
}

// The staged tile's first `rows` rows, `bytes` of each, to y (row pitch in bytes).
// vec: y and the pitch are multiples of 16 bytes, and so is `bytes`; otherwise
// elements of ES bytes go one by one.
template <int ROWB, int ES>
__device__ __forceinline__ void stage_flush(const uint8_t* buf, uint8_t* y, int64_t pitch, int rows, int bytes, bool vec,
                                            int lane) {
  if (vec) {
    constexpr int PER = ROWB / 16, RPI = 32 / PER;  // lanes per row, rows per instruction
    const int c = lane % PER;
    uint8_t* dst = y + (int64_t)(lane / PER) * pitch + c * 16;
    if (rows >= 32 && bytes >= ROWB) {
#pragma unroll
      for (int r = 0; r < 32; r += RPI) {
        const uint4 q = *reinterpret_cast<const uint4*>(buf + stage_off<ROWB>((uint32_t)(r + lane / PER), (uint32_t)c));
        *reinterpret_cast<uint4*>(dst + (int64_t)r * pitch) = q;
      }
    } else {
#pragma unroll 1
      for (int r = lane / PER; r < rows; r += RPI)
        if (c * 16 < bytes)
          *reinterpret_cast<uint4*>(y + (int64_t)r * pitch + c * 16) =
              *reinterpret_cast<const uint4*>(buf + stage_off<ROWB>((uint32_t)r, (uint32_t)c));
    }
  } else {  // neighbouring lanes on neighbouring elements of one row
    constexpr int PER = ROWB / ES < 32 ? ROWB / ES : 32, RPI = 32 / PER;  // lanes per row, rows per instruction
#pragma unroll 4
    for (int r = lane / PER; r < rows; r += RPI) {
#pragma unroll
      for (int e = 0; e < ROWB; e += PER * ES) {
        const int b = e + (lane % PER) * ES;
        const uint8_t* src = buf + stage_off<ROWB>((uint32_t)r, (uint32_t)(b >> 4)) + (b & 15);
        if (b < bytes) {
          if constexpr (ES == 4)
            *reinterpret_cast<uint32_t*>(y + (int64_t)r * pitch + b) = *reinterpret_cast<const uint32_t*>(src);
          else
            *reinterpret_cast<uint16_t*>(y + (int64_t)r * pitch + b) = *reinterpret_cast<const uint16_t*>(src);
        }
      }
    }
  }
}

}  // namespace nm

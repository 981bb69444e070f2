// nm_stage.cuh -- output staging of the kernels whose accumulator lanes are
// output rows: each thread of a warp holds a run of one row's columns; the warp's
// 32 rows go through a small swizzled buffer in shared memory and leave as one
// tensor store (or, where the row pitch rules that out, as plain stores along
// the rows).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nm_device.cuh"

namespace nm {

__host__ __device__ constexpr int stage_elem_bytes(int ot) { return ot == OUT_F32 ? 4 : 2; }

// Byte offset of 16-byte piece c of row `row` in a staged tile with rows of
// ROWB bytes: the tensor store's swizzle of that width (address bits 4.. of a
// 16-byte piece XOR bits 7..), which also spreads a warp's 16-byte writes over
// all banks (rows of 32 bytes: two per bank).
template <int ROWB>
__device__ __forceinline__ uint32_t stage_off(uint32_t row, uint32_t c) {
  static_assert(ROWB == 128 || ROWB == 64 || ROWB == 32, "swizzle widths");
  const uint32_t x = ROWB == 128 ? (row & 7u) : ROWB == 64 ? ((row >> 1) & 3u) : ((row >> 2) & 1u);
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

// NV values of this thread's row into the staged tile.
template <int OT, int NV>
__device__ __forceinline__ void stage_row(uint8_t* buf, uint32_t row, const float* v) {
  constexpr int ROWB = NV * stage_elem_bytes(OT);
#pragma unroll
  for (int c = 0; c < ROWB / 16; ++c) {
    uint4 q;
    if constexpr (OT == OUT_F32) {
      q = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                     __float_as_uint(v[4 * c + 3]));
    } else {
      q = make_uint4(pack_pair<OT>(v[8 * c], v[8 * c + 1]), pack_pair<OT>(v[8 * c + 2], v[8 * c + 3]),
                     pack_pair<OT>(v[8 * c + 4], v[8 * c + 5]), pack_pair<OT>(v[8 * c + 6], v[8 * c + 7]));
    }
    *reinterpret_cast<uint4*>(buf + stage_off<ROWB>(row, (uint32_t)c)) = q;
  }
}

// The staged tile's first `rows` rows and `cols` columns to y (row pitch ld
// elements) by plain stores, neighbouring lanes on neighbouring columns.
template <int OT, int NV>
__device__ __forceinline__ void stage_copy_rows(const uint8_t* buf, void* y, int64_t ld, int rows, int cols,
                                                int lane) {
  constexpr int ES = stage_elem_bytes(OT), ROWB = NV * ES, PER = 16 / ES, RPI = 32 / NV;
  const int col = lane % NV;
  for (int r = lane / NV; r < rows; r += RPI) {
    const uint8_t* src = buf + stage_off<ROWB>((uint32_t)r, (uint32_t)(col / PER)) + (col % PER) * ES;
    if (col < cols) {
      if constexpr (ES == 4)
        reinterpret_cast<uint32_t*>(y)[r * ld + col] = *reinterpret_cast<const uint32_t*>(src);
      else
        reinterpret_cast<uint16_t*>(y)[r * ld + col] = *reinterpret_cast<const uint16_t*>(src);
    }
  }
}

}  // namespace nm

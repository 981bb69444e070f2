// nm_unpack.cuh -- element access shared by the packing kernels and the kernels
// that read a packed weight back.
#pragma once
#include "nm_device.cuh"

namespace nm {

template <int DT>
struct Elem;
template <>
struct Elem<DT_I8> {
  using T = int8_t;
  __device__ static uint32_t mag(T v) { return (uint32_t)(v < 0 ? -(int)v : (int)v); }
};
template <int DT>
struct Elem {  // FP16 / BF16 as raw bits: |x| orders like the bits with the sign cleared
  using T = uint16_t;
  __device__ static uint32_t mag(T v) { return (uint32_t)(v & 0x7FFFu); }
};

// 16 bytes <-> elements, little-endian, without type punning local arrays.
template <typename T>
__device__ __forceinline__ uint4 pack16(const T* v) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
  for (int e = 0; e < 16 / (int)sizeof(T); ++e) {
    const uint32_t bits = sizeof(T) == 1 ? (uint32_t)(uint8_t)v[e] : (uint32_t)(uint16_t)v[e];
    w[e / per] |= bits << (8 * (int)sizeof(T) * (e % per));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void unpack16(uint4 q, T* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
  for (int e = 0; e < 16 / (int)sizeof(T); ++e) {
    const uint32_t bits = w[e / per] >> (8 * (int)sizeof(T) * (e % per));
    v[e] = sizeof(T) == 1 ? (T)(int8_t)(uint8_t)bits : (T)(uint16_t)bits;
  }
}

// 16 consecutive dense k positions (k0 a multiple of 16) of W's row r, decoded from
// the packed image into Wout [rows][K].  n_ff > 0: a gated weight.  (Coherent loads: the
// image may come from the kernel just before.)
template <int DT>
__device__ __forceinline__ void unpack_unit(const uint8_t* __restrict__ bpack, int64_t n_ff, int64_t K, int img, int n_kb,
                                            typename Elem<DT>::T* __restrict__ Wout, int64_t r, int64_t k0) {
  using T = typename Elem<DT>::T;
  constexpr int KB = kblock_elems(DT);
  constexpr int ES = elem_bytes(DT);
  const int valid = (int)(K - k0 > 16 ? 16 : K - k0);
  const int64_t pr = n_ff ? gated_packed_row(r, n_ff) : r;
  const int64_t ct = pr / kRows;
  const uint32_t rr = (uint32_t)(pr % kRows);
  const int kb = (int)(k0 / KB);
  const uint32_t kk = (uint32_t)(k0 % KB);
  const uint8_t* chunk = bpack + ((size_t)ct * n_kb + kb) * (size_t)chunk_bytes(DT, img);

  T out[16];
  if (img == IMG_SP24) {
    T comp[8];
    if (ES == 1) {
      const unsigned long long v = ld_coherent(reinterpret_cast<const unsigned long long*>(chunk + swz128(rr, kk / 2)));
#pragma unroll
      for (int e = 0; e < 8; ++e) comp[e] = (T)(int8_t)(uint8_t)(v >> (8 * e));
    } else {
      unpack16<T>(ld_coherent(reinterpret_cast<const uint4*>(chunk + swz128(rr, kk))), comp);
    }
    const uint32_t meta = ld_coherent(reinterpret_cast<const uint16_t*>(chunk + kAtomBytes + meta_off16(DT, rr, kk)));
    // positions of a group's two slots always differ; selects keep `out` in registers
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int nib = (meta >> (4 * j)) & 0xF;
      const int i0 = nib & 3, i1 = (nib >> 2) & 3;
#pragma unroll
      for (int c = 0; c < 4; ++c) out[4 * j + c] = c == i0 ? comp[2 * j] : c == i1 ? comp[2 * j + 1] : (T)0;
    }
  } else {
#pragma unroll
    for (int h = 0; h < ES; ++h) {
      const uint32_t byte = kk * ES + 16u * h;
      unpack16<T>(ld_coherent(reinterpret_cast<const uint4*>(chunk + (byte >> 7) * kAtomBytes + swz128(rr, byte & 127u))),
                  out + h * (16 / ES));
    }
  }
  T* dst = Wout + r * K + k0;
  if (valid == 16 && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
#pragma unroll
    for (int h = 0; h < ES; ++h) reinterpret_cast<uint4*>(dst)[h] = pack16<T>(out + h * (16 / ES));
  } else {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (c < valid) dst[c] = out[c];
  }
}

}  // namespace nm

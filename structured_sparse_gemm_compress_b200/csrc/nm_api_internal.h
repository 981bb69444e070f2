// nm_api_internal.h -- what the files that implement the C ABI share: error
// reporting, device queries and argument checks (defined in nm_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "nmspmm.h"
#include "nm_internal.h"

namespace nm {

void clear_error();
// Record the message of the calling thread's failing call and return `st`.
nm_status fail(nm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
nm_status cuda_fail(cudaError_t e, const char* what);
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int num_sms(int dev);
// NM_ERR_INVALID for a null handle or one of another device than the current one.
nm_status check_handle(const nm_handle* h);
// Whether the library prunes to N:M (sp24: on the 2:4 sparse tensor core).
bool pattern_supported(int N, int M, bool* sp24);
// One device allocation for several buffers of a handle: sizes are added first,
// then allocated, then handed out in the same order (256-byte aligned).
struct Arena {
  size_t total = 0;
  uint8_t* base = nullptr;
  size_t add(size_t bytes) {
    const size_t at = total;
    total += (bytes + 255) / 256 * 256;
    return at;
  }
  cudaError_t allocate(nm_handle* h) {
    cudaError_t e = cudaMalloc(&h->d_arena, total);
    base = static_cast<uint8_t*>(h->d_arena);
    return e;
  }
};
// [a, a + an) and [b, b + bn) share a byte.
inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// A tiled tensor map over `rank` dimensions (innermost first; strides in bytes
// of dimensions 1 ..), zero fill outside the tensor.
nm_status encode_map(CUtensorMap* map, CUtensorMapDataType ty, int rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle,
                     CUtensorMapL2promotion promotion);

// Output stage of one call after nm_epilogue has been checked.
struct EpiReq {
  int out_ty = -1;  // nm::OUT_F32 / F16 / BF16 / I8
  const float* bias = nullptr;
  int act = ACT_NONE;
  float out_scale = 1.0f;
};

}  // namespace nm

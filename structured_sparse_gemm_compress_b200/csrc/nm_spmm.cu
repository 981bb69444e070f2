// nm_spmm.cu -- host side of the N:M SpMM kernels (nm_spmm_kernels.cuh): the
// instances of the ungated products, their dispatch, and how many clusters of
// each can be resident.
#include "nm_spmm_kernels.cuh"

namespace nm {

int pair_max_clusters(int dt, int img, int bn, int out);

template <int DT, int IMG, int OUT>
static cudaError_t launch_bn(const CUtensorMap* tmX, const CUtensorMap* tmY, const CUtensorMap* tmW,
                             const Plan& p, const SpmmArgs& a, cudaStream_t s) {
  if (p.pair) {
    switch (p.bn) {
      case 128: return launch_pair_t<DT, IMG, 128, OUT>(tmX, tmY, tmW, p, a, s);
      case 192: return launch_pair_t<DT, IMG, 192, OUT>(tmX, tmY, tmW, p, a, s);
      case 224: return launch_pair_t<DT, IMG, 224, OUT>(tmX, tmY, tmW, p, a, s);
      default: return cudaErrorInvalidValue;
    }
  }
  if (p.xkb > 0) {  // X-stationary mode: INT8, 128-token tiles, up to kXsMaxKb k-blocks (k <= 768)
    if constexpr (DT == DT_I8) {
      if (p.bn == 128 && p.xkb <= kXsMaxKb) return launch_t<DT, IMG, 128, OUT, kXsMaxKb>(tmX, tmY, tmW, p, a, s);
    }
    return cudaErrorInvalidValue;
  }
  switch (p.bn) {
    case 32: return launch_t<DT, IMG, 32, OUT, 0>(tmX, tmY, tmW, p, a, s);
    case 64: return launch_t<DT, IMG, 64, OUT, 0>(tmX, tmY, tmW, p, a, s);
    case 128: return launch_t<DT, IMG, 128, OUT, 0>(tmX, tmY, tmW, p, a, s);
    case 192: return launch_t<DT, IMG, 192, OUT, 0>(tmX, tmY, tmW, p, a, s);
    default: return cudaErrorInvalidValue;
  }
}

// Gather image: streaming kernel only, direct-store output stages (fixed or runtime).
template <int DT, int OUT>
static cudaError_t launch_gather(const CUtensorMap* tmX, const CUtensorMap* tmY, const CUtensorMap* tmW,
                                 const Plan& p, const SpmmArgs& a, cudaStream_t s) {
  if constexpr (DT != DT_BF16 && (OUT & kOutDirect) != 0) {
    if (p.pair || p.xkb > 0) return cudaErrorInvalidValue;
    switch (p.bn) {
      case 128: return launch_t<DT, IMG_GATHER, 128, OUT, 0>(tmX, tmY, tmW, p, a, s);
      case 256: return launch_t<DT, IMG_GATHER, 256, OUT, 0>(tmX, tmY, tmW, p, a, s);
      default: return cudaErrorInvalidValue;
    }
  }
  return cudaErrorInvalidValue;
}

template <int DT, int OUT>
static cudaError_t launch_img(int img, const CUtensorMap* tmX, const CUtensorMap* tmY, const CUtensorMap* tmW,
                              const Plan& p, const SpmmArgs& a, cudaStream_t s) {
  if (img == IMG_GATHER) return launch_gather<DT, OUT>(tmX, tmY, tmW, p, a, s);
  return img == IMG_SP24 ? launch_bn<DT, IMG_SP24, OUT>(tmX, tmY, tmW, p, a, s)
                         : launch_bn<DT, IMG_DENSE, OUT>(tmX, tmY, tmW, p, a, s);
}

template <int OUT_TS>
static cudaError_t launch_dt(const nm_handle* h, const CUtensorMap* tmX, const CUtensorMap* tmY,
                             const CUtensorMap* tmW, const Plan& p, const SpmmArgs& a, cudaStream_t s) {
  constexpr int D = OUT_TS;  // 0 or kOutDirect
  if constexpr (D == kOutDirect) {
    if (a.out_ty >= 0) {  // runtime output stage
      switch (h->dt) {
        case DT_I8: return launch_img<DT_I8, kOutEpi | kOutDirect>(h->img, tmX, tmY, tmW, p, a, s);
        case DT_F16: return launch_img<DT_F16, kOutEpi | kOutDirect>(h->img, tmX, tmY, tmW, p, a, s);
        default: return launch_img<DT_BF16, kOutEpi | kOutDirect>(h->img, tmX, tmY, tmW, p, a, s);
      }
    }
  } else {
    if (a.out_ty >= 0) return cudaErrorInvalidValue;  // the runtime output stage stores directly
  }
  switch (h->dt) {
    case DT_I8:
      return a.scale ? launch_img<DT_I8, OUT_F32 | D>(h->img, tmX, tmY, tmW, p, a, s)
                     : launch_img<DT_I8, OUT_I32 | D>(h->img, tmX, tmY, tmW, p, a, s);
    case DT_F16: return launch_img<DT_F16, OUT_F16 | D>(h->img, tmX, tmY, tmW, p, a, s);
    default: return launch_img<DT_BF16, OUT_BF16 | D>(h->img, tmX, tmY, tmW, p, a, s);
  }
}

cudaError_t launch_spmm(const nm_handle* h, const CUtensorMap* tmX, const CUtensorMap* tmY, const Plan& p,
                        const SpmmArgs& a, cudaStream_t s) {
  const CUtensorMap* tmW = &h->tmw;
  return a.tma_store ? launch_dt<0>(h, tmX, tmY, tmW, p, a, s) : launch_dt<kOutDirect>(h, tmX, tmY, tmW, p, a, s);
}

// Pairs that can be resident at once for a pair-kernel configuration (cached per device).
template <int DT, int IMG, int BN, int OUT>
static int max_clusters_t() {
  static std::atomic<int> cache[64];
  static std::atomic<uint64_t> opted{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  int cached = cache[dev].load(std::memory_order_acquire);
  if (!cached) {
    using C = PairCfg<DT, IMG, BN, OUT>;
    auto kern = spmm_pair_kernel<DT, IMG, BN, OUT>;
    if (smem_opt_in(kern, C::SMEM, opted) != cudaSuccess) cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.attrs = nullptr;  // the kernel declares its cluster shape (2 CTAs) at compile time
    cfg.numAttrs = 0;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (void*)kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
    cached = n > 0 ? n : -1;
    cache[dev].store(cached, std::memory_order_release);
  }
  return cached;
}

int stream_max_clusters(int size) {
  static std::atomic<int> cache[64][kMaxClusterSplit + 1];
  static std::atomic<uint64_t> opted{0};
  int dev = 0;
  if (size < 1 || size > kMaxClusterSplit) return -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  int cached = cache[dev][size].load(std::memory_order_acquire);
  if (!cached) {
    // every streaming configuration runs one CTA per SM, so one instance answers for all
    using C = Cfg<DT_I8, IMG_SP24, 32, OUT_I32 | kOutDirect, 0>;
    auto kern = spmm_kernel<DT_I8, IMG_SP24, 32, OUT_I32 | kOutDirect, 0>;
    if (smem_opt_in(kern, C::SMEM, opted) != cudaSuccess) cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size, 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (void*)kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
    cached = n > 0 ? n : -1;
    cache[dev][size].store(cached, std::memory_order_release);
  }
  return cached;
}

int pair_max_clusters(int dt, int img, int bn, int out) {
  // All configurations share threads and (nearly) shared memory: one query per dtype/bn suffices.
  int n = -1;
  if (dt == DT_I8) {
    const bool f32 = out == OUT_F32;
    if (img == IMG_SP24) n = bn == 224 ? (f32 ? max_clusters_t<DT_I8, IMG_SP24, 224, OUT_F32>() : max_clusters_t<DT_I8, IMG_SP24, 224, OUT_I32>())
                       : bn == 192 ? (f32 ? max_clusters_t<DT_I8, IMG_SP24, 192, OUT_F32>() : max_clusters_t<DT_I8, IMG_SP24, 192, OUT_I32>())
                                   : (f32 ? max_clusters_t<DT_I8, IMG_SP24, 128, OUT_F32>() : max_clusters_t<DT_I8, IMG_SP24, 128, OUT_I32>());
    else n = bn == 224 ? (f32 ? max_clusters_t<DT_I8, IMG_DENSE, 224, OUT_F32>() : max_clusters_t<DT_I8, IMG_DENSE, 224, OUT_I32>())
           : bn == 192 ? (f32 ? max_clusters_t<DT_I8, IMG_DENSE, 192, OUT_F32>() : max_clusters_t<DT_I8, IMG_DENSE, 192, OUT_I32>())
                       : (f32 ? max_clusters_t<DT_I8, IMG_DENSE, 128, OUT_F32>() : max_clusters_t<DT_I8, IMG_DENSE, 128, OUT_I32>());
  } else if (dt == DT_F16) {
    n = img == IMG_SP24 ? (bn == 224 ? max_clusters_t<DT_F16, IMG_SP24, 224, OUT_F16>() : bn == 192 ? max_clusters_t<DT_F16, IMG_SP24, 192, OUT_F16>() : max_clusters_t<DT_F16, IMG_SP24, 128, OUT_F16>())
                        : (bn == 224 ? max_clusters_t<DT_F16, IMG_DENSE, 224, OUT_F16>() : bn == 192 ? max_clusters_t<DT_F16, IMG_DENSE, 192, OUT_F16>() : max_clusters_t<DT_F16, IMG_DENSE, 128, OUT_F16>());
  } else {
    n = img == IMG_SP24 ? (bn == 224 ? max_clusters_t<DT_BF16, IMG_SP24, 224, OUT_BF16>() : bn == 192 ? max_clusters_t<DT_BF16, IMG_SP24, 192, OUT_BF16>() : max_clusters_t<DT_BF16, IMG_SP24, 128, OUT_BF16>())
                        : (bn == 224 ? max_clusters_t<DT_BF16, IMG_DENSE, 224, OUT_BF16>() : bn == 192 ? max_clusters_t<DT_BF16, IMG_DENSE, 192, OUT_BF16>() : max_clusters_t<DT_BF16, IMG_DENSE, 128, OUT_BF16>());
  }
  return n;
}

}  // namespace nm

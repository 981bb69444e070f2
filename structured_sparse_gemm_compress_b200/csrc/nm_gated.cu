// nm_gated.cu -- the instances of the N:M SpMM kernels with the gated output stage
// (nm_spmm_gated): the streaming kernel, unsplit or split over a cluster, and
// the two-SM kernel, for every element type and weight image.
#include "nm_spmm_kernels.cuh"

namespace nm {
namespace {

constexpr int kOut = kOutEpi | kOutDirect | kOutGate;

template <int DT, int IMG>
cudaError_t launch_img(const CUtensorMap* tmX, const CUtensorMap* tmW, const Plan& p, const SpmmArgs& a,
                       cudaStream_t s) {
  // the output never leaves by tensor stores: its map argument is not read
  if (p.xkb > 0 || (p.splits > 1 && !p.cluster)) return cudaErrorInvalidValue;
  if (p.pair) {
    if constexpr (DT != DT_I8) {
      if (a.P && a.n_ff % 8 == 0) {  // every row of p starts on 16 bytes
        if (p.bn == 192) return launch_pair_t<DT, IMG, 192, kOut | kOutSave>(tmX, tmX, tmW, p, a, s);
        if (p.bn == 128) return launch_pair_t<DT, IMG, 128, kOut | kOutSave>(tmX, tmX, tmW, p, a, s);
        return cudaErrorInvalidValue;
      }
    }
    if (p.bn == 192) return launch_pair_t<DT, IMG, 192, kOut>(tmX, tmX, tmW, p, a, s);
    if (p.bn == 128) return launch_pair_t<DT, IMG, 128, kOut>(tmX, tmX, tmW, p, a, s);
    return cudaErrorInvalidValue;
  }
  switch (p.bn) {
    case 32: return launch_t<DT, IMG, 32, kOut, 0>(tmX, tmX, tmW, p, a, s);
    case 64: return launch_t<DT, IMG, 64, kOut, 0>(tmX, tmX, tmW, p, a, s);
    case 128: return launch_t<DT, IMG, 128, kOut, 0>(tmX, tmX, tmW, p, a, s);
    case 192:  // the dense image leaves two stages at this tile: the planner does not use it
      if constexpr (IMG == IMG_SP24) return launch_t<DT, IMG, 192, kOut, 0>(tmX, tmX, tmW, p, a, s);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

template <int DT>
cudaError_t launch_dt(const nm_handle* h, const CUtensorMap* tmX, const Plan& p, const SpmmArgs& a, cudaStream_t s) {
  return h->img == IMG_SP24 ? launch_img<DT, IMG_SP24>(tmX, &h->tmw, p, a, s)
                            : launch_img<DT, IMG_DENSE>(tmX, &h->tmw, p, a, s);
}

}  // namespace

cudaError_t launch_spmm_gated(const nm_handle* h, const CUtensorMap& tmX, const Plan& p, const SpmmArgs& a,
                              cudaStream_t s) {
  switch (h->dt) {
    case DT_I8: return launch_dt<DT_I8>(h, &tmX, p, a, s);
    case DT_F16: return launch_dt<DT_F16>(h, &tmX, p, a, s);
    default: return launch_dt<DT_BF16>(h, &tmX, p, a, s);
  }
}

}  // namespace nm

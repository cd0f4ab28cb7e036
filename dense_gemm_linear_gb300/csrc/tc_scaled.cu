// Instantiations of the tcgen05 tile kernel whose elements are scaled by one factor.
#include "tc_launch.cuh"

namespace dgl {

namespace {

template <int BN, int CG>
cudaError_t launch(int out, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tbh, const CUtensorMap& tc,
                   const TcParams& p, int grid, cudaStream_t stream) {
  return out == 1 ? tc_launch_one<BN, false, true, false, CG, false, false, 128, 3>(ta, tb, tbh, tc, p, grid, stream)
                  : tc_launch_one<BN, false, false, false, CG, false, false, 128, 3>(ta, tb, tbh, tc, p, grid, stream);
}

}  // namespace

cudaError_t launch_tc_scaled(int out, int tile_m, int tile_n, const CUtensorMap& ta, const CUtensorMap& tb,
                             const CUtensorMap& tbh, const CUtensorMap& tc, const TcParams& p, int grid,
                             cudaStream_t stream) {
  if (tile_m == 256 && tile_n == 256) return launch<256, 2>(out, ta, tb, tbh, tc, p, grid, stream);
  if (tile_m == 256 && tile_n == 128) return launch<128, 2>(out, ta, tb, tbh, tc, p, grid, stream);
  if (tile_m == 128 && tile_n == 256) return launch<256, 1>(out, ta, tb, tbh, tc, p, grid, stream);
  if (tile_m == 128 && tile_n == 128) return launch<128, 1>(out, ta, tb, tbh, tc, p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace dgl

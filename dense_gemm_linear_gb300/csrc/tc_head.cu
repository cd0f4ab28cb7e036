// Instantiations of the tcgen05 tile kernel with the epilogue of a linear head's logits.
#include "tc_launch.cuh"

namespace dgl {

namespace {

template <int HEAD>
cudaError_t launch(int tile_m, int tile_n, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                   const TcParams& p, int grid, cudaStream_t stream) {
  if (tile_m == 256 && tile_n == 256)
    return tc_launch_one<256, false, false, false, 2, false, false, 128, HEAD>(ta, tb, tb, tc, p, grid, stream);
  if (tile_m == 128 && tile_n == 256)
    return tc_launch_one<256, false, false, false, 1, false, false, 128, HEAD>(ta, tb, tb, tc, p, grid, stream);
  if (tile_m == 128 && tile_n == 128)
    return tc_launch_one<128, false, false, false, 1, false, false, 128, HEAD>(ta, tb, tb, tc, p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tc_head(bool store, int tile_m, int tile_n, const CUtensorMap& ta, const CUtensorMap& tb,
                           const CUtensorMap& tc, const TcParams& p, int grid, cudaStream_t stream) {
  return store ? launch<2>(tile_m, tile_n, ta, tb, tc, p, grid, stream)
               : launch<1>(tile_m, tile_n, ta, tb, tc, p, grid, stream);
}

}  // namespace dgl

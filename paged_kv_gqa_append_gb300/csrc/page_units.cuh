// The (row, layer) pairs of a release shared out over warps (page_stack.cu).  On its own, so that it
// also compiles for the host, where a test goes through sizes that need many GiB of tables.
#pragma once

namespace pkv {

// Warp `warp` of `warps` takes the pairs warp, warp + warps, ... of the list (0, 0), (0, 1), ...; there
// may be more of them (4096 rows of 2^30 layers) than 32 bits hold, so row and layer are kept apart.
struct UnitWalk {
  int row, layer, rows_on, layers_on, layers;
  __device__ __forceinline__ UnitWalk(int warp, int warps, int layers_)
      : row(warp / layers_), layer(warp % layers_), rows_on(warps / layers_), layers_on(warps % layers_), layers(layers_) {}
  __device__ __forceinline__ void next() {  // (both layers are below 2^30)
    row += rows_on;
    layer += layers_on;
    if (layer >= layers) {
      layer -= layers;
      ++row;
    }
  }
};

}  // namespace pkv

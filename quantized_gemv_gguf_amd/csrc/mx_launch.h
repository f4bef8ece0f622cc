// mx_launch.h -- which kernel of mx_gemm.h a product takes, by sizes and type.
#pragma once

#include "mx_gemm.h"

namespace qgemv_mx {

// Places an expert gets on average decide the tile.
template <int XK>
hipError_t launch_mx(const MxArgs &a, hipStream_t stream) {
  const int64_t avg = a.offsets ? (a.places + a.n_expert - 1) / a.n_expert : a.places;
  if (a.w2) {
    if (avg <= 16) return launch_tile<XK, true, 1, 1, 4, 1>(a, stream);
    return launch_tile<XK, true, 2, 4, 4, 1>(a, stream);
  }
  if (avg <= 16) return launch_tile<XK, false, 2, 1, 4, 1>(a, stream);
  return launch_tile<XK, false, 2, 4, 4, 1>(a, stream);
}

}  // namespace qgemv_mx

// kv_attend_launch.h -- the attention kernels of one cache type, by head size.
#pragma once

#include "kv_attend.h"

namespace qgemv_kv {

// f(first, count) for all workgroups, a launch at a time.
template <typename F> void in_grids(int64_t groups, F f) {
  for (int64_t first = 0; first < groups; first += kMaxGrid)
    f(first, dim3((unsigned)(groups - first < kMaxGrid ? groups - first : kMaxGrid)));
}

template <int T, int D, int NT> void launch_rows(const AttendArgs &a, const AttendShape &s, hipStream_t stream) {
  const bool few = s.rows == kFewRows;
  in_grids(s.parts * a.kv_heads, [&](int64_t first, dim3 grid) {
    if (few) hipLaunchKernelGGL((attend_few_kernel<T, D, NT>), grid, dim3(64 * FewTile<D>::kWaves), 0, stream, a, first);
    else hipLaunchKernelGGL((attend_many_kernel<T, D, NT>), grid, dim3(64 * kManyWaves), 0, stream, a, first);
  });
  if (a.target == 0) return;
  // few tiles are joined by many workgroups
  const int rows = few ? s.tiles * a.kv_heads <= 128 ? 1 : 16 : s.tiles * a.kv_heads <= 128 ? 16 : kManyRows;
  in_grids(s.tiles * (s.rows / rows) * a.kv_heads, [&](int64_t first, dim3 grid) {
    if (few)
      hipLaunchKernelGGL((attend_join_kernel<D, kFewRows, kFewPiece>), grid, dim3(256), 0, stream, a, rows, first);
    else
      hipLaunchKernelGGL((attend_join_kernel<D, kManyRows, kManyPiece>), grid, dim3(256), 0, stream, a, rows, first);
  });
}

template <int T, int D> void launch_dim(const AttendArgs &a, const AttendShape &s, bool wide, hipStream_t stream) {
  if (wide) launch_rows<T, D, Kind<T>::kWide>(a, s, stream);
  else launch_rows<T, D, 1>(a, s, stream);
}

template <int T>
hipError_t launch_attend(const AttendArgs &a, const AttendShape &s, int dim, bool wide, hipStream_t stream) {
  switch (dim) {
    case 32: launch_dim<T, 32>(a, s, wide, stream); break;
    case 64: launch_dim<T, 64>(a, s, wide, stream); break;
    case 96: launch_dim<T, 96>(a, s, wide, stream); break;
    case 128: launch_dim<T, 128>(a, s, wide, stream); break;
    case 160: launch_dim<T, 160>(a, s, wide, stream); break;
    case 192: launch_dim<T, 192>(a, s, wide, stream); break;
    case 224: launch_dim<T, 224>(a, s, wide, stream); break;
    default: launch_dim<T, 256>(a, s, wide, stream); break;
  }
  return hipGetLastError();
}

}  // namespace qgemv_kv

// mx_launch.h -- which kernel of mx_gemm.h a product takes.
#pragma once

#include "mx_gemm.h"

namespace qgemv_mx {

constexpr double kNever = 1e300;  // the time of a grid that cannot be launched

// A tile shape with its measured times, in 0.1 us at k = 4096: kOne, a grid of
// at most one workgroup per compute unit; kMore, each further workgroup per
// compute unit.  kWhole: one workgroup at a time fills a compute unit (LDS or
// registers), so a grid takes whole rounds.
template <int XK, bool PAIR, int FN, int FM, int WN, int WM, int WK, int KS, int NBUF, int kOne, int kMore, bool kWhole,
          bool COLS = false>
struct Shape {
  using S = MxTile<XK, PAIR, FN, FM, WN, WM, WK, KS, NBUF, COLS>;

  // Estimated time; tokens are taken as spread evenly over the experts, each
  // adding a partial tile of 0.6 (0.5, and unevenness: 4096 MXFP4 tokens x 4 of
  // 128 experts of 2880 x 2880 take tiles of 128 tokens with it, 277 us, not of
  // 256, 317).
  static double cost(const MxArgs &a) {
    if (!Grid<S>(a).fits()) return kNever;
    const double active = a.offsets ? (a.n_expert < a.places ? a.n_expert : a.places) : 1;
    const double each = a.places / active;
    double tm = a.offsets ? (each + 0.6 * S::TM) / S::TM : (double)((a.places - 1) / S::TM + 1);
    if (tm < 1.0) tm = 1.0;
    double per_cu = active * tm * ((a.n - 1) / S::TN + 1) / 256.0;
    if (kWhole) per_cu = (double)(int64_t)(per_cu + 0.999);
    // whole stages, and a workgroup's start and end (measured: the time of 0.3
    // to 1.1 stages, of the largest 0.8 to 2.6)
    constexpr double kEnds = kWhole ? 1.5 : 0.7;
    const double length = ((a.nb + S::kBlk - 1) / S::kBlk + kEnds) / (128.0 / S::kBlk + kEnds);
    return (kOne + (per_cu > 1.0 ? (per_cu - 1.0) * kMore : 0.0)) * length;
  }
  static hipError_t launch(const MxArgs &a, hipStream_t stream) {
    return launch_tile<XK, PAIR, FN, FM, WN, WM, WK, KS, NBUF, COLS>(a, stream);
  }
};

// Of several shapes the one with the least estimated time.  Timed against every
// shape of its kind for 37 problems each (1 to 4096 tokens, dense, and of 8 to 147
// experts; k = 64 to 12480), the chosen one took 1.01 times the best (geometric
// mean; 1.3 to 1.4 in three calls of 9 to 17 us).  No one shape does: bf16 tokens, 5 x
// 11008 outputs of k = 4096, 13 us in the smallest shape and 56 in the largest;
// 2048 x 8192, 805 and 134.
template <typename... Of>
struct Cheapest {
  static constexpr int kShapes = sizeof...(Of);
  static int best(const MxArgs &a) {  // -1 if no shape's grid holds the product
    const double costs[] = {Of::cost(a)...};
    int at = 0;
    for (int i = 1; i < kShapes; ++i)
      if (costs[i] < costs[at]) at = i;
    return costs[at] < kNever ? at : -1;
  }
  static int stage_blocks(int shape) {  // blocks of a row that a stage takes
    const int blocks[] = {Of::S::kBlk...};
    return blocks[shape];
  }
  static hipError_t run(const MxArgs &a, hipStream_t stream, bool *fits) {
    hipError_t (*const launches[])(const MxArgs &, hipStream_t) = {Of::launch...};
    const int shape = best(a);
    *fits = shape >= 0;
    return *fits ? launches[shape](a, stream) : hipSuccess;
  }
};

template <int XK, bool PAIR> struct Shapes;

template <>
struct Shapes<kFp4, false>
    : Cheapest<Shape<kFp4, false, 2, 1, 1, 1, 4, 4, 2, 52, 19, false>,
               Shape<kFp4, false, 2, 2, 1, 1, 4, 4, 2, 68, 28, false>,
               Shape<kFp4, false, 2, 4, 2, 1, 2, 4, 1, 125, 62, false>,
               Shape<kFp4, false, 4, 4, 4, 2, 1, 2, 2, 285, 270, true>,
               Shape<kFp4, false, 4, 8, 4, 2, 1, 2, 2, 415, 430, true>> {};
template <>
struct Shapes<kFp4, true>
    : Cheapest<Shape<kFp4, true, 1, 1, 1, 1, 4, 4, 2, 60, 23, false>,
               Shape<kFp4, true, 1, 2, 1, 1, 4, 4, 2, 65, 25, false>,
               Shape<kFp4, true, 1, 4, 2, 1, 2, 4, 1, 115, 56, false>,
               Shape<kFp4, true, 1, 4, 4, 1, 1, 2, 1, 160, 97, false>,
               Shape<kFp4, true, 2, 4, 4, 2, 1, 2, 2, 270, 275, true>,
               Shape<kFp4, true, 2, 8, 4, 2, 1, 2, 2, 445, 450, true>> {};
template <>
struct Shapes<kBf16, false>
    : Cheapest<Shape<kBf16, false, 2, 1, 1, 1, 8, 8, 2, 72, 62, true>,
               Shape<kBf16, false, 2, 2, 4, 1, 1, 2, 1, 210, 130, false>,
               Shape<kBf16, false, 2, 4, 8, 1, 1, 1, 2, 335, 365, true>,
               Shape<kBf16, false, 4, 4, 4, 2, 1, 1, 2, 560, 610, true>> {};
template <>
struct Shapes<kBf16, true>
    : Cheapest<Shape<kBf16, true, 1, 1, 1, 1, 8, 8, 2, 62, 60, true>,
               Shape<kBf16, true, 1, 1, 2, 1, 4, 4, 1, 88, 60, false>,
               Shape<kBf16, true, 1, 2, 4, 1, 1, 2, 1, 200, 120, false>,
               Shape<kBf16, true, 2, 2, 8, 2, 1, 1, 2, 620, 670, true>,
               Shape<kBf16, true, 4, 3, 4, 2, 1, 1, 2, 770, 830, true>> {};
template <>
struct Shapes<kF16, false>
    : Cheapest<Shape<kF16, false, 1, 1, 1, 1, 8, 8, 1, 44, 28, false, true>,
               Shape<kF16, false, 2, 1, 1, 1, 8, 8, 1, 52, 41, true, true>,
               Shape<kF16, false, 2, 2, 4, 1, 1, 2, 1, 300, 195, false>,
               Shape<kF16, false, 8, 2, 4, 2, 1, 1, 2, 900, 1080, true>> {};
template <>
struct Shapes<kF16, true>
    : Cheapest<Shape<kF16, true, 1, 1, 1, 1, 8, 8, 1, 66, 38, false, true>,
               Shape<kF16, true, 1, 1, 2, 1, 4, 4, 1, 118, 58, false, true>,
               Shape<kF16, true, 1, 2, 4, 1, 1, 2, 1, 296, 180, false>,
               Shape<kF16, true, 2, 4, 8, 1, 1, 1, 2, 1000, 1000, true>> {};
template <>
struct Shapes<kF32, false>
    : Cheapest<Shape<kF32, false, 1, 1, 1, 1, 8, 8, 1, 44, 28, false, true>,
               Shape<kF32, false, 2, 1, 1, 1, 8, 8, 1, 55, 40, true, true>,
               Shape<kF32, false, 2, 1, 1, 1, 8, 8, 1, 97, 115, true>,
               Shape<kF32, false, 2, 1, 4, 1, 1, 2, 1, 260, 145, false>,
               Shape<kF32, false, 4, 2, 4, 2, 1, 1, 2, 850, 850, true>,
               Shape<kF32, false, 4, 2, 8, 2, 1, 1, 1, 1250, 1350, true>> {};
template <>
struct Shapes<kF32, true>
    : Cheapest<Shape<kF32, true, 1, 1, 1, 1, 8, 8, 1, 72, 42, false, true>,
               Shape<kF32, true, 1, 1, 1, 1, 4, 4, 1, 80, 36, false, true>,
               Shape<kF32, true, 1, 1, 2, 1, 4, 4, 1, 125, 64, false, true>,
               Shape<kF32, true, 1, 1, 2, 1, 4, 4, 1, 130, 112, true>,
               Shape<kF32, true, 1, 1, 4, 1, 1, 2, 1, 305, 152, false>,
               Shape<kF32, true, 1, 2, 4, 1, 1, 1, 1, 435, 247, false>,
               Shape<kF32, true, 2, 2, 4, 2, 1, 1, 2, 730, 730, true>,
               Shape<kF32, true, 2, 1, 8, 2, 1, 1, 2, 750, 750, true>> {};

template <int XK>
hipError_t launch_mx(const MxArgs &a, hipStream_t stream, bool *fits) {
  return a.w2 ? Shapes<XK, true>::run(a, stream, fits) : Shapes<XK, false>::run(a, stream, fits);
}

}  // namespace qgemv_mx

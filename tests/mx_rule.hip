// Which shape of mx_launch.h a product takes: reads "kind pair places rows blocks
// experts" lines (kind: bf16 terms, 0 for MXFP4; experts 0: dense) and prints the
// shape, the shapes there are and the blocks of one of its stages.  Host code only.
#include <stdio.h>

#include "mx_launch.h"

using namespace qgemv_mx;

template <int XK, bool PAIR>
static void print(const MxArgs &a) {
  using S = Shapes<XK, PAIR>;
  const int at = S::best(a);
  printf("%d %d %d\n", at, S::kShapes, at < 0 ? 0 : S::stage_blocks(at));
}

template <int XK>
static void print(const MxArgs &a, int pair) {
  if (pair) print<XK, true>(a);
  else print<XK, false>(a);
}

int main() {
  const int32_t some = 0;
  int kind, pair, n_expert;
  MxArgs a = {};
  while (scanf("%d %d %d %d %d %d", &kind, &pair, &a.places, &a.n, &a.nb, &n_expert) == 6) {
    a.n_expert = n_expert > 0 ? n_expert : 1;
    a.offsets = n_expert > 0 ? &some : nullptr;
    if (kind == kF32) print<kF32>(a, pair);
    else if (kind == kF16) print<kF16>(a, pair);
    else if (kind == kBf16) print<kBf16>(a, pair);
    else print<kFp4>(a, pair);
  }
}

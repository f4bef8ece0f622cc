// mx_bf16.hip -- products of bf16 activations with MXFP4 weights (mx_gemm.h).
#include "mx_launch.h"

namespace qgemv_mx {
template hipError_t launch_mx<kBf16>(const MxArgs &a, hipStream_t stream, bool *fits);
}

// mx_f16.hip -- products of f16 activations with MXFP4 weights (mx_gemm.h).
#include "mx_launch.h"

namespace qgemv_mx {
template hipError_t launch_mx<kF16>(const MxArgs &a, hipStream_t stream, bool *fits);
}

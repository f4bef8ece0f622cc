// mx_fp4.hip -- products of MXFP4 activations with MXFP4 weights (mx_gemm.h).
#include "mx_launch.h"

namespace qgemv_mx {
template hipError_t launch_mx<kFp4>(const MxArgs &a, hipStream_t stream, bool *fits);
}

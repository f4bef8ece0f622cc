// kv_attend_bf16.hip -- attention over a cache of bf16 keys and values (kv_attend.h).
#include "kv_attend_launch.h"

namespace qgemv_kv {
template hipError_t launch_attend<QG_BF16>(const AttendArgs &a, const AttendShape &s, int dim, bool wide,
                                        hipStream_t stream);
}

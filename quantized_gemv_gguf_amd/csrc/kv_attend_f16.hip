// kv_attend_f16.hip -- attention over a cache of f16 keys and values (kv_attend.h).
#include "kv_attend_launch.h"

namespace qgemv_kv {
template hipError_t launch_attend<QG_F16>(const AttendArgs &a, const AttendShape &s, int dim, bool wide,
                                        hipStream_t stream);
}

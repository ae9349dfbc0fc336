// The attention over a cache of bf16 rows.
#include "attend_kernel.h"

namespace fp4 {
hipError_t launch_attend_bf16(const AttendParams& p, hipStream_t s) { return attend::launch_parts<kStoreBf16>(p, s); }
}  // namespace fp4

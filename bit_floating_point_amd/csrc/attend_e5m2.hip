// The attention over a cache of E5M2 codes.
#include "attend_kernel.h"

namespace fp4 {
hipError_t launch_attend_e5m2(const AttendParams& p, hipStream_t s) { return attend::launch_parts<kStoreE5m2>(p, s); }
}  // namespace fp4

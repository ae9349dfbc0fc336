// The attention over a cache of E2M1 codes.
#include "attend_kernel.h"

namespace fp4 {
hipError_t launch_attend_e2m1(const AttendParams& p, hipStream_t s) { return attend::launch_parts<kStoreE2m1>(p, s); }
}  // namespace fp4

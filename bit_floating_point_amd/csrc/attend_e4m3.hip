// The attention over a cache of E4M3 codes.
#include "attend_kernel.h"

namespace fp4 {
hipError_t launch_attend_e4m3(const AttendParams& p, hipStream_t s) { return attend::launch_parts<kStoreE4m3>(p, s); }
}  // namespace fp4

// Linear attention's walk for f16 elements.
#include "linattn.h"

namespace symnmf {
template hipError_t launch_attend_walk<f16_t>(const AttendArgs&, bool, hipStream_t);
}

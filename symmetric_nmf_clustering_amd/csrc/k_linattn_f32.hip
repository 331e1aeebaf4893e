// Linear attention's walk for f32 elements.
#include "linattn.h"

namespace symnmf {
template hipError_t launch_attend_walk<float>(const AttendArgs&, bool, hipStream_t);
}

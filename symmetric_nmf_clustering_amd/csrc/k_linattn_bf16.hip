// Linear attention's walk for bf16 elements.
#include "linattn.h"

namespace symnmf {
template hipError_t launch_attend_walk<bf16_t>(const AttendArgs&, bool, hipStream_t);
}

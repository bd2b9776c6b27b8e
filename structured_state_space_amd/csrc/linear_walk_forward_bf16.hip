// The forward walk of linear attention, bf16 activations.
// (An instance of the __global__ templates of linear_walk.hpp.)
#include "linear_walk.hpp"

namespace ssm {
template hipError_t launch_walk<bf16, false>(const WalkArgs&, hipStream_t);
}  // namespace ssm

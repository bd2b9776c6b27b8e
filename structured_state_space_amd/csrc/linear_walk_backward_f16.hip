// The backward walk of linear attention, f16 activations.
// (An instance of the __global__ templates of linear_walk.hpp.)
#include "linear_walk.hpp"

namespace ssm {
template hipError_t launch_walk<f16, true>(const WalkArgs&, hipStream_t);
}  // namespace ssm

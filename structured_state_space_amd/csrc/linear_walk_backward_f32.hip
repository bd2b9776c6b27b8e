// The backward walk of linear attention, f32 activations.
// (An instance of the __global__ templates of linear_walk.hpp.)
#include "linear_walk.hpp"

namespace ssm {
template hipError_t launch_walk<float, true>(const WalkArgs&, hipStream_t);
}  // namespace ssm

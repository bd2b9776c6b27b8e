// The gradients of linear attention, f16 activations.
// (An instance of the __global__ templates of linear_grad.hpp.)
#include "linear_grad.hpp"

namespace ssm {
template hipError_t launch_pairs<f16>(const PairArgs&, hipStream_t);
}  // namespace ssm

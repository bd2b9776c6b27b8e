// Argument blocks of the layer norm kernels.
#pragma once

#include "linear.hpp"

namespace ssm {

struct NormArgs {
    int64_t Bsz, H, L, G;
    int rms, gate;
    float eps;
    View3 u, z, y;  // z.data null without a gate
    const float *weight, *bias;  // [H] nullable
};
struct NormGradArgs {
    NormArgs f;  // the forward call's (y unused)
    View3 dy, du, dz;
    float *dweight, *dbias;  // [H] nullable
    float* parts;            // [2, rows, H]: sums of dweight and dbias over some of the steps; null without both
    int64_t rows;
};

// 1 / sqrt(v): the hardware's (one unit; it takes subnormal numbers for zero) and one step of Newton's method
__device__ __forceinline__ float inverse_root(float v) {
    const bool low = v < 0x1p-126f;
    v *= low ? 0x1p24f : 1.0f;
    float r = __builtin_amdgcn_rsqf(v);
    const float e = fmaf(-v * r, r, 1.0f);
    r = fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
    return r * (low ? 0x1p12f : 1.0f);
}

// the grid of the kernel that the views select; whether either order's gradients have one for these sizes
bool norm_fits(const NormArgs& a);
bool norm_fits(const NormGradArgs& g);
bool norm_grad_may_fit(int64_t Bsz, int64_t L, int64_t D, int64_t G);
int64_t norm_part_rows(int64_t Bsz, int64_t L, int64_t D, int64_t G);
hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(int dtype, NormGradArgs& g, hipStream_t s);

}  // namespace ssm

// Linear attention of one token per sequence (include/ssm.h: ssm_linear_attention_step).
#include "linear.hpp"

namespace ssm {

constexpr int kTokenThreads = 256;
constexpr int kTokenValues = 64;
constexpr int kTokenAhead = 8;  // vectors of the state that a thread has under way

// A workgroup has one head of a sequence, and of its values up to 64: the state is read
// once, moved on by a step, written back and multiplied with the query on the way.  A
// thread keeps to V neighbouring values, so that its part of the product stays in
// registers; the threads of the same values add theirs in LDS.  Bound by the state's 8
// bytes per element: 250 sequences of 64 heads, 128 keys, 64 values, 198 us, 5.3 TB/s.
// (Sixteen values to a workgroup where the heads are few: 32 heads 4.9 us instead of 4.2, 256
// heads 10 instead of 5.2; the state's rows are then read 64 bytes at a time.)
template <class T, int V>
__global__ __launch_bounds__(kTokenThreads) void linear_step_kernel(const LinearStepArgs a) {
    struct __attribute__((packed, aligned(4))) Vec { float v[V]; };
    __shared__ float ks[kMaxKeys], qs[kMaxKeys], part[kTokenThreads * V];
    const int tid = threadIdx.x, N = (int)a.N, P = (int)a.P;
    const int blocks = (P + kTokenValues - 1) / kTokenValues;
    const int pb = (int)(blockIdx.x % blocks), h = (int)(blockIdx.x / blocks % a.H);
    const int64_t b = (int64_t)blockIdx.x / blocks / a.H;
    int64_t row = b;
    if (a.slots) {
        row = a.slots[b];
        if (row < 0 || row >= a.n_slots) return;
    }
    const int grp = (int)(h / (a.H / a.G));
    const float beta = a.beta ? a.beta[b * a.beta_row + h * a.beta_head] : 1.0f;
    // (weights above one come last: beta k must not pass float32 where the value is zero, nor scale q where
    // the state is)
    const float first = fabsf(beta) <= 1.0f ? beta : 1.0f, last = fabsf(beta) <= 1.0f ? 1.0f : beta;
    const float q_first = fabsf(a.scale) <= 1.0f ? a.scale : 1.0f, q_last = fabsf(a.scale) <= 1.0f ? 1.0f : a.scale;
    const float e = exp_f<kFine<T>>(a.g[b * a.g_row + h * a.g_head]);
    const int p0 = pb * kTokenValues, wide = min(kTokenValues, P - p0) / V;  // vectors of a row
    const int rows = kTokenThreads / wide, r = tid / wide, p = p0 + tid % wide * V;
    const bool live = r < rows;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f(((const T*)a.v)[b * a.v_row + h * a.v_head + (p + i) * a.v_value]);
    for (int n = tid; n < N; n += kTokenThreads) {
        ks[n] = first * to_f(((const T*)a.k)[b * a.k_row + grp * a.k_group + n * a.k_key]);
        qs[n] = q_first * to_f(((const T*)a.q)[b * a.q_row + grp * a.q_group + n * a.q_key]);
    }
    __syncthreads();
    float* x = a.x + ((row * a.H + h) * N) * P + p;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = 0.0f;
    if (live)
        for (int n0 = r; n0 < N; n0 += rows * kTokenAhead) {
            Vec s[kTokenAhead];
#pragma unroll
            for (int j = 0; j < kTokenAhead; ++j) {
                const int n = n0 + j * rows;
                if (n < N) s[j] = *reinterpret_cast<const Vec*>(x + (int64_t)n * P);
            }
#pragma unroll
            for (int j = 0; j < kTokenAhead; ++j) {
                const int n = n0 + j * rows;
                if (n < N) {
                    const float k = ks[n], q = qs[n];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s[j].v[i] = fmaf(s[j].v[i], e, k * v[i] * last);
                        y[i] = fmaf(s[j].v[i], q, y[i]);
                    }
                    *reinterpret_cast<Vec*>(x + (int64_t)n * P) = s[j];
                }
            }
        }
    if (live) {
#pragma unroll
        for (int i = 0; i < V; ++i) part[(r * wide + tid % wide) * V + i] = y[i];
    }
    __syncthreads();
    for (int c = tid; c < wide * V; c += kTokenThreads) {
        float sum = 0.0f;
        for (int k = 0; k < rows; ++k) sum += part[k * wide * V + c];
        sum *= q_last;
        if (a.D) sum = fmaf(a.D[h], to_f(((const T*)a.v)[b * a.v_row + h * a.v_head + (p0 + c) * a.v_value]), sum);
        ((T*)a.y)[b * a.y_row + h * a.y_head + (p0 + c) * a.y_value] = from_f<T>(sum);
    }
}

static int64_t token_workgroups(int64_t Bsz, int64_t H, int64_t P) { return Bsz * H * ((P + kTokenValues - 1) / kTokenValues); }

template <class T>
static void launch(const LinearStepArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)token_workgroups(a.Bsz, a.H, a.P)), wg(kTokenThreads);
    if (a.P % 4 == 0) hipLaunchKernelGGL((linear_step_kernel<T, 4>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((linear_step_kernel<T, 1>), grid, wg, 0, s, a);
}

bool linear_step_fits(int64_t Bsz, int64_t H, int64_t P) { return grid_fits(token_workgroups(Bsz, H, P), kTokenThreads); }

hipError_t launch_linear_step(int dtype, const LinearStepArgs& a, hipStream_t s) {
    if (dtype == SSM_F32) launch<float>(a, s);
    else if (dtype == SSM_BF16) launch<bf16>(a, s);
    else launch<f16>(a, s);
    return hipGetLastError();
}

}  // namespace ssm

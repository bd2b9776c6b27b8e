// Single-token forms of the selective operators, for decoding on states that
// live in a pool: sequence b's state is row slots[b] (b without slots); a slot
// outside the pool names no state, and its sequence is left alone.
//
//   selective step   x <- exp(dt A) x + dt u B,  y = (sum_n C[n] x[n] + D u) silu(z)
//   convolution step y = act(bias + sum_k w[k] line[k]), line = state then u;
//                    the state moves on by one
//
// Both are bound by the state's bytes, read and written once: 8 N bytes per
// channel for the scan.  A quad of lanes holds a channel's states, four (16
// bytes) per lane and block of 16, so a wave reads whole lines; a workgroup has 64
// channels of one sequence.  250 sequences of 4096 channels, N = 16, bf16: 29 us,
// 4.7 TB/s, what a large copy reaches (with four sequences to a workgroup, A read once
// for them, 32 us); one sequence of 2048 channels: 3.4 us, a launch's own time and one
// trip to memory.  The convolution, 250 x 8192, width 4, f16: 11 us, 3.0 TB/s.
#include "selective.hpp"

namespace ssm {

namespace {

// states 16 nb + 4 q + j of one channel; W4: 16-byte accesses (N a multiple of 4, aligned)
template <bool W4>
__device__ __forceinline__ void load_states(float (&r)[4], const float* p, int n0, int N) {
    if (W4) {
        if (n0 < N) {
            const float4 v = *reinterpret_cast<const float4*>(p + n0);
            r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
        } else {
            r[0] = r[1] = r[2] = r[3] = 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = n0 + j < N ? p[n0 + j] : 0.0f;
    }
}
template <bool W4>
__device__ __forceinline__ void store_states(const float (&r)[4], float* p, int n0, int N) {
    if (W4) {
        if (n0 < N) *reinterpret_cast<float4*>(p + n0) = make_float4(r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + j < N) p[n0 + j] = r[j];
    }
}

template <class T, int NB, bool W4>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a, int blocks) {
    const int64_t cb = blockIdx.x % blocks, b = blockIdx.x / blocks;
    const int q = threadIdx.x & 3, N = (int)a.N;
    const int64_t h = cb * 64 + (threadIdx.x >> 2);
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    if (h >= a.H || slot < 0 || slot >= a.n_slots) return;
    const int64_t g = h / (a.H / a.G);
    const bool dense = a.B_state == 1 && a.C_state == 1;
    float x[NB][4], bv[NB][4], cv[NB][4], A2[NB][4];
    float* const state = a.x + (slot * a.H + h) * N;
    const float u = to_f(((const T*)a.u)[b * a.u_row + h]);
    const float dt = to_f(((const T*)a.delta)[b * a.delta_row + h]);
    const float z = a.z ? to_f(((const T*)a.z)[b * a.z_row + h]) : 0.0f;
    const T* Bp = (const T*)a.B + b * a.B_row + g * a.B_group;
    const T* Cp = (const T*)a.C + b * a.C_row + g * a.C_group;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int n0 = nb * 16 + q * 4;
        load_states<W4>(x[nb], state, n0, N);
        load_states<W4>(A2[nb], a.A + h * N, n0, N);
        if (dense && n0 + 4 <= N) {
            const Vec4<T> vb = *reinterpret_cast<const Vec4<T>*>(Bp + n0);
            const Vec4<T> vc = *reinterpret_cast<const Vec4<T>*>(Cp + n0);
#pragma unroll
            for (int j = 0; j < 4; ++j) bv[nb][j] = to_f(vb.v[j]), cv[nb][j] = to_f(vc.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bv[nb][j] = n0 + j < N ? to_f(Bp[(n0 + j) * a.B_state]) : 0.0f;
                cv[nb][j] = n0 + j < N ? to_f(Cp[(n0 + j) * a.C_state]) : 0.0f;
            }
        }
    }
    const float bias = a.delta_bias ? a.delta_bias[h] : 0.0f, D = a.D ? a.D[h] : 0.0f;
    const float v = dt + bias, s = a.softplus ? softplus_f<kFine<T>>(v) : v, dx = s * u;
    float y = 0.0f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[nb][j] = fmaf(__builtin_amdgcn_exp2f(s * (A2[nb][j] * kLog2e)), x[nb][j], dx * bv[nb][j]);
            // (behind the last state 0, also where dt u is infinite)
            y = fmaf(cv[nb][j], nb * 16 + q * 4 + j < N ? x[nb][j] : 0.0f, y);
        }
        store_states<W4>(x[nb], state, nb * 16 + q * 4, N);
    }
    y += dpp<0xB1>(y);
    y += dpp<0x4E>(y);
    if (q == 0) {
        y = fmaf(D, u, y);
        if (a.z) y *= silu_f<kFine<T>>(z);
        ((T*)a.y)[b * a.y_row + h] = from_f<T>(y);
    }
}

// V channels of one sequence per thread; their states are V (W - 1) consecutive elements
template <class T, int W, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a, int64_t per_row) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = i / per_row, h = (i % per_row) * V;
    if (b >= a.Bsz) return;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    if (slot < 0 || slot >= a.n_slots) return;
    const int n = (int)min((int64_t)V, a.H - h);
    T* st = (T*)a.state + (slot * a.H + h) * (W - 1);
    const T* u = (const T*)a.u + b * a.u_row + h;
    T* y = (T*)a.y + b * a.y_row + h;
    struct __attribute__((packed, aligned(sizeof(T)))) Line {
        T v[W > 1 ? V * (W - 1) : 1];
    };
    struct __attribute__((packed, aligned(sizeof(T)))) Out {
        T v[V];
    };
    struct __attribute__((packed, aligned(4))) Weights {
        float v[V * W];
    };
    if (n == V) {
        Line line;
        if (W > 1) line = *reinterpret_cast<const Line*>(st);
        const Out in = *reinterpret_cast<const Out*>(u);
        const Weights w = *reinterpret_cast<const Weights*>(a.weight + h * W);
        Out out;
        Line next;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            float acc = a.bias ? a.bias[h + c] : 0.0f;
#pragma unroll
            for (int k = 0; k < W - 1; ++k) acc = fmaf(w.v[c * W + k], to_f(line.v[c * (W - 1) + k]), acc);
            acc = fmaf(w.v[c * W + W - 1], to_f(in.v[c]), acc);
            out.v[c] = from_f<T>(a.silu ? silu_f<kFine<T>>(acc) : acc);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                next.v[c * (W - 1) + k] = k + 1 < W - 1 ? line.v[c * (W - 1) + (k + 1 < W - 1 ? k + 1 : 0)] : in.v[c];
        }
        if (W > 1) *reinterpret_cast<Line*>(st) = next;
        *reinterpret_cast<Out*>(y) = out;
    } else {
        for (int c = 0; c < n; ++c) {
            float acc = a.bias ? a.bias[h + c] : 0.0f;
            T* s = st + c * (W - 1);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) acc = fmaf(a.weight[(h + c) * W + k], to_f(s[k]), acc);
            acc = fmaf(a.weight[(h + c) * W + W - 1], to_f(u[c]), acc);
            y[c] = from_f<T>(a.silu ? silu_f<kFine<T>>(acc) : acc);
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) s[k] = s[k + 1];
            if (W > 1) s[W > 1 ? W - 2 : 0] = u[c];
        }
    }
}

template <class T, int NB, bool W4>
hipError_t step_as(const StepArgs& a, hipStream_t s) {
    const int64_t blocks = (a.H + 63) / 64, wgs = a.Bsz * blocks;
    if (!grid_fits(wgs, 256)) return hipErrorInvalidValue;
    step_kernel<T, NB, W4><<<dim3((unsigned)wgs), dim3(256), 0, s>>>(a, (int)blocks);
    return hipGetLastError();
}

template <class T>
hipError_t step_of(const StepArgs& a, hipStream_t s) {
    const bool w4 = a.N % 4 == 0 && (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.A % 16 == 0;
    if (a.N <= 16) return w4 ? step_as<T, 1, true>(a, s) : step_as<T, 1, false>(a, s);
    if (a.N <= 32) return w4 ? step_as<T, 2, true>(a, s) : step_as<T, 2, false>(a, s);
    return w4 ? step_as<T, 4, true>(a, s) : step_as<T, 4, false>(a, s);
}

template <class T, int W>
hipError_t conv_step_as(const ConvStepArgs& a, hipStream_t s) {
    constexpr int V = 4;
    const int64_t per_row = (a.H + V - 1) / V, wgs = (a.Bsz * per_row + 255) / 256;
    if (!grid_fits(wgs, 256)) return hipErrorInvalidValue;
    conv_step_kernel<T, W, V><<<dim3((unsigned)wgs), dim3(256), 0, s>>>(a, per_row);
    return hipGetLastError();
}

template <class T>
hipError_t conv_step_of(const ConvStepArgs& a, hipStream_t s) {
    switch (a.width) {
        case 1: return conv_step_as<T, 1>(a, s);
        case 2: return conv_step_as<T, 2>(a, s);
        case 3: return conv_step_as<T, 3>(a, s);
        default: return conv_step_as<T, 4>(a, s);
    }
}

}  // namespace

hipError_t launch_selective_step(int dtype, const StepArgs& a, hipStream_t s) {
    if (dtype == SSM_F32) return step_of<float>(a, s);
    if (dtype == SSM_BF16) return step_of<bf16>(a, s);
    return step_of<f16>(a, s);
}

hipError_t launch_causal_conv_step(int dtype, const ConvStepArgs& a, hipStream_t s) {
    if (dtype == SSM_F32) return conv_step_of<float>(a, s);
    if (dtype == SSM_BF16) return conv_step_of<bf16>(a, s);
    return conv_step_of<f16>(a, s);
}

}  // namespace ssm

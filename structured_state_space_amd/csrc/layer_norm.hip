// Layer norm over groups of channels, with or without the mean and a gate, and its
// gradients (include/ssm.h: ssm_layer_norm).
#include "norm.hpp"

namespace ssm {

struct Stats {
    float mean, scale;  // 1 / sqrt(variance + eps)
};
__device__ __forceinline__ float wave_sum(float v) { return across_rows(row_sum(v)); }

// what the norm sees of an element, and how its gradient goes back
template <class T>
__device__ __forceinline__ float gated(float u, float z, int gate) {
    return gate == SSM_GATE_BEFORE ? u * silu_f<kFine<T>>(z) : u;
}
// d silu(z) / dz
template <class T>
__device__ __forceinline__ float silu_slope(float z) {
    const float p = sigmoid_f<kFine<T>>(z);
    return p * fmaf(z, 1.0f - p, 1.0f);
}

// ---- channels contiguous ----
// LANES threads have the channels of a group at one step, eight neighbours to a vector, V
// vectors each: the step's numbers are read once, stay in registers between the sums (the
// mean first, then the squares about it) and are written once.  Bound by memory.
template <int LANES>
__device__ __forceinline__ float group_sum(float v, float* part) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    if constexpr (LANES > 8) v += dpp<0x140>(v);
    if constexpr (LANES > 16) v += __shfl_xor(v, 16);
    if constexpr (LANES > 32) v += __shfl_xor(v, 32);
    if constexpr (LANES > 64) {
        __syncthreads();  // the last sum has been read
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < LANES / 64; ++i) v += part[i];
    }
    return v;
}
template <class T>
__device__ __forceinline__ void load8(float (&r)[8], const void* data, int64_t at, int there) {
    const T* p = (const T*)data + at;
    if (there >= 8) {
        const Vec8<T> w = *reinterpret_cast<const Vec8<T>*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = to_f(w.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = i < there ? to_f(p[i]) : 0.0f;
    }
}
template <class T>
__device__ __forceinline__ void store8(const float (&r)[8], const void* data, int64_t at, int there) {
    T* p = (T*)data + at;
    if (there >= 8) {
        Vec8<T> w;
#pragma unroll
        for (int i = 0; i < 8; ++i) w.v[i] = from_f<T>(r[i]);
        *reinterpret_cast<Vec8<T>*>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < there) p[i] = from_f<T>(r[i]);
    }
}
constexpr int norm_threads(int lanes) { return lanes > 256 ? lanes : 256; }

template <class T, int LANES, int V>
__global__ __launch_bounds__(norm_threads(LANES)) void norm_rows_kernel(const NormArgs a) {
    constexpr int R = norm_threads(LANES) / LANES;  // steps of a workgroup
    __shared__ float part[LANES > 64 ? LANES / 64 : 1];
    const int tid = threadIdx.x, D = (int)(a.H / a.G);
    const int64_t row = (int64_t)blockIdx.x * R + tid / LANES;  // (batch row, step, group)
    if (row >= a.Bsz * a.L * a.G) return;
    const int grp = (int)(row % a.G);
    const int64_t l = row / a.G % a.L, b = row / a.G / a.L;
    const int first = tid % LANES * 8;
    float x[V][8], z[V][8];
    int there[V];
    const int64_t u0 = b * a.u.sb + l * a.u.sl + grp * D, z0 = b * a.z.sb + l * a.z.sl + grp * D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = first + v * LANES * 8;
        there[v] = D - c;
        load8<T>(x[v], a.u.data, u0 + c, there[v]);
        if (a.gate) load8<T>(z[v], a.z.data, z0 + c, there[v]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (a.gate == SSM_GATE_BEFORE) x[v][i] = i < there[v] ? gated<T>(x[v][i], z[v][i], a.gate) : 0.0f;
            sum += x[v][i];
        }
    const float mean = a.rms ? 0.0f : group_sum<LANES>(sum, part) / (float)D;
    float squares = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[v][i] = i < there[v] ? x[v][i] - mean : 0.0f;
            squares = fmaf(x[v][i], x[v][i], squares);
        }
    const float scale = inverse_root(group_sum<LANES>(squares, part) / (float)D + a.eps);
    const int64_t y0 = b * a.y.sb + l * a.y.sl + grp * D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = first + v * LANES * 8;
        if (there[v] <= 0) continue;
        float w[8], s[8], y[8];
        if (a.weight) load8<float>(w, a.weight, grp * D + c, there[v]);
        if (a.bias) load8<float>(s, a.bias, grp * D + c, there[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = x[v][i] * scale;
            y[i] = a.weight ? (a.bias ? fmaf(n, w[i], s[i]) : n * w[i]) : (a.bias ? n + s[i] : n);
            if (a.gate == SSM_GATE_AFTER) y[i] *= silu_f<kFine<T>>(z[v][i]);
        }
        store8<T>(y, a.y.data, y0 + c, there[v]);
    }
}

// Gradients.  With n the normed numbers and dn = dy' weight (dy' behind a gate on the output):
//   da = (dn - mean dn - n mean(dn n)) / sqrt(variance + eps)
// (without mean dn where the mean was not taken), dweight = sum dy' n, dbias = sum dy'.
// The norm is computed again: its numbers are in registers, and the call takes nothing from
// the forward pass.  Workgroups go over steps `rows` apart with the same channels in the same
// lanes, so that the parameters' sums stay in registers until the end; each then has a row
// of partial sums.
template <class T, int LANES, int V>
__global__ __launch_bounds__(norm_threads(LANES)) void norm_rows_grad_kernel(const NormGradArgs g) {
    const NormArgs& a = g.f;
    constexpr int R = norm_threads(LANES) / LANES;
    __shared__ float part[LANES > 64 ? LANES / 64 : 1];
    const int tid = threadIdx.x, D = (int)(a.H / a.G);
    const int grp = (int)(blockIdx.x % a.G);
    const int64_t mine = (int64_t)(blockIdx.x / a.G) * R + tid / LANES;
    const int first = tid % LANES * 8;
    const int64_t steps = a.Bsz * a.L;
    float dw[V][8], db[V][8], w[V][8], s[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = first + v * LANES * 8, there = D - c;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = db[v][i] = 0.0f, w[v][i] = 1.0f, s[v][i] = 0.0f;
        if (a.weight) load8<float>(w[v], a.weight, grp * D + c, there);
        if (a.bias && a.gate == SSM_GATE_AFTER) load8<float>(s[v], a.bias, grp * D + c, there);
    }
    for (int64_t r = mine; r < steps; r += g.rows) {
        const int64_t l = r % a.L, b = r / a.L;
        const int64_t u0 = b * a.u.sb + l * a.u.sl + grp * D, z0 = b * a.z.sb + l * a.z.sl + grp * D;
        const int64_t y0 = b * g.dy.sb + l * g.dy.sl + grp * D;
        float u[V][8], z[V][8], d[V][8], n[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = first + v * LANES * 8, there = D - c;
            load8<T>(u[v], a.u.data, u0 + c, there);
            if (a.gate) load8<T>(z[v], a.z.data, z0 + c, there);
            load8<T>(d[v], g.dy.data, y0 + c, there);
        }
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = first + v * LANES * 8 + i < D;
                n[v][i] = a.gate == SSM_GATE_BEFORE ? (in ? gated<T>(u[v][i], z[v][i], a.gate) : 0.0f) : u[v][i];
                sum += n[v][i];
            }
        const float mean = a.rms ? 0.0f : group_sum<LANES>(sum, part) / (float)D;
        float squares = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[v][i] = first + v * LANES * 8 + i < D ? n[v][i] - mean : 0.0f;
                squares = fmaf(n[v][i], n[v][i], squares);
            }
        const float scale = inverse_root(group_sum<LANES>(squares, part) / (float)D + a.eps);
        float m0 = 0.0f, m1 = 0.0f;
        const int64_t dz0 = b * g.dz.sb + l * g.dz.sl + grp * D;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = first + v * LANES * 8, there = D - c;
            float dz[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[v][i] *= scale;
                if (a.gate == SSM_GATE_AFTER) {
                    dz[i] = d[v][i] * fmaf(n[v][i], w[v][i], s[v][i]) * silu_slope<T>(z[v][i]);
                    d[v][i] = i < there ? d[v][i] * silu_f<kFine<T>>(z[v][i]) : 0.0f;
                }
                dw[v][i] = fmaf(d[v][i], n[v][i], dw[v][i]);
                db[v][i] += d[v][i];
                d[v][i] *= w[v][i];
                m0 += d[v][i];
                m1 = fmaf(d[v][i], n[v][i], m1);
            }
            if (a.gate == SSM_GATE_AFTER && there > 0) store8<T>(dz, g.dz.data, dz0 + c, there);
        }
        const float c0 = a.rms ? 0.0f : group_sum<LANES>(m0, part) / (float)D;
        const float c1 = group_sum<LANES>(m1, part) / (float)D;
        const int64_t du0 = b * g.du.sb + l * g.du.sl + grp * D;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = first + v * LANES * 8, there = D - c;
            if (there <= 0) continue;
            float du[8], dz[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                du[i] = scale * (d[v][i] - c0 - n[v][i] * c1);
                if (a.gate == SSM_GATE_BEFORE) {
                    dz[i] = du[i] * u[v][i] * silu_slope<T>(z[v][i]);
                    du[i] *= silu_f<kFine<T>>(z[v][i]);
                }
            }
            store8<T>(du, g.du.data, du0 + c, there);
            if (a.gate == SSM_GATE_BEFORE) store8<T>(dz, g.dz.data, dz0 + c, there);
        }
    }
    if (g.parts) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = first + v * LANES * 8, there = D - c;
            if (there <= 0) continue;
            store8<float>(dw[v], g.parts, mine * a.H + grp * D + c, there);
            store8<float>(db[v], g.parts, (g.rows + mine) * a.H + grp * D + c, there);
        }
    }
}

// ---- any other order: 64 steps to a workgroup, a lane each ----
// A lane takes its step's channels in blocks of kBlock, whose loads fly together; the waves
// share the channels.  Means and squares are joined block by block (the squares about the
// joined mean: m2 + m2' + delta^2 n n' / (n + n')), so that the numbers are read twice.
constexpr int kStepThreads = 512;
constexpr int kStepWaves = kStepThreads / 64;
constexpr int kBlock = 16;

struct Running {
    float count = 0.0f, mean = 0.0f, m2 = 0.0f;
    __device__ __forceinline__ void join(float n, float mu, float q) {
        const float all = count + n, share = n / all, delta = mu - mean;
        mean = fmaf(delta, share, mean);
        m2 += q + delta * delta * count * share;
        count = all;
    }
};
template <class T>
__device__ __forceinline__ Stats step_stats(const NormArgs& a, const T* u, const T* z, int D, bool live, int wave, int lane,
                                            float (*parts)[3][64]) {
    Running s;
    for (int c0 = wave * kBlock; c0 < D; c0 += kStepWaves * kBlock) {
        float x[kBlock];
        const int n = min(kBlock, D - c0);
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            x[i] = 0.0f;
            if (live && i < n) {
                x[i] = to_f(u[(c0 + i) * a.u.sh]);
                if (a.gate == SSM_GATE_BEFORE) x[i] = gated<T>(x[i], to_f(z[(c0 + i) * a.z.sh]), a.gate);
            }
        }
        float sum = 0.0f, squares = 0.0f;
        if (!a.rms) {
#pragma unroll
            for (int i = 0; i < kBlock; ++i) sum += x[i];
        }
        const float mean = sum / (float)n;
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            const float d = i < n ? x[i] - mean : 0.0f;
            squares = fmaf(d, d, squares);
        }
        s.join((float)n, mean, squares);
    }
    parts[wave][0][lane] = s.count, parts[wave][1][lane] = s.mean, parts[wave][2][lane] = s.m2;
    __syncthreads();
    Running all;
#pragma unroll
    for (int i = 0; i < kStepWaves; ++i)
        if (parts[i][0][lane] > 0.0f) all.join(parts[i][0][lane], parts[i][1][lane], parts[i][2][lane]);
    __syncthreads();
    return {all.mean, inverse_root(all.m2 / (float)D + a.eps)};
}

template <class T>
__global__ __launch_bounds__(kStepThreads) void norm_steps_kernel(const NormArgs a, int64_t blocks) {
    __shared__ float parts[kStepWaves][3][64];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int D = (int)(a.H / a.G), grp = (int)(blockIdx.x % a.G);
    const int64_t l = blockIdx.x / a.G % blocks * 64 + lane, b = blockIdx.x / a.G / blocks;
    const bool live = l < a.L;
    const int64_t at = live ? l : a.L - 1;
    const T* u = (const T*)a.u.data + b * a.u.sb + at * a.u.sl + (int64_t)grp * D * a.u.sh;
    const T* z = a.gate ? (const T*)a.z.data + b * a.z.sb + at * a.z.sl + (int64_t)grp * D * a.z.sh : nullptr;
    T* y = (T*)a.y.data + b * a.y.sb + at * a.y.sl + (int64_t)grp * D * a.y.sh;
    const Stats s = step_stats<T>(a, u, z, D, live, wave, lane, parts);
    if (!live) return;
    for (int c0 = wave * kBlock; c0 < D; c0 += kStepWaves * kBlock) {
        float x[kBlock], e[kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i)
            if (c0 + i < D) {
                x[i] = to_f(u[(c0 + i) * a.u.sh]);
                if (a.gate) e[i] = to_f(z[(c0 + i) * a.z.sh]);
            }
#pragma unroll
        for (int i = 0; i < kBlock; ++i)
            if (c0 + i < D) {
                const int c = grp * D + c0 + i;
                const float n = ((a.gate == SSM_GATE_BEFORE ? gated<T>(x[i], e[i], a.gate) : x[i]) - s.mean) * s.scale;
                float v = fmaf(n, a.weight ? a.weight[c] : 1.0f, a.bias ? a.bias[c] : 0.0f);
                if (a.gate == SSM_GATE_AFTER) v *= silu_f<kFine<T>>(e[i]);
                y[(c0 + i) * a.y.sh] = from_f<T>(v);
            }
    }
}

// Gradients: the two means in a second pass, the rest in a third; a channel's sums over the
// 64 steps are sums over the lanes.
template <class T>
__global__ __launch_bounds__(kStepThreads) void norm_steps_grad_kernel(const NormGradArgs g, int64_t blocks) {
    const NormArgs& a = g.f;
    __shared__ float parts[kStepWaves][3][64];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int D = (int)(a.H / a.G), grp = (int)(blockIdx.x % a.G);
    const int64_t block = blockIdx.x / a.G, l = block % blocks * 64 + lane, b = block / blocks;
    const bool live = l < a.L;
    const int64_t at = live ? l : a.L - 1;
    const T* u = (const T*)a.u.data + b * a.u.sb + at * a.u.sl + (int64_t)grp * D * a.u.sh;
    const T* z = a.gate ? (const T*)a.z.data + b * a.z.sb + at * a.z.sl + (int64_t)grp * D * a.z.sh : nullptr;
    const T* dy = (const T*)g.dy.data + b * g.dy.sb + at * g.dy.sl + (int64_t)grp * D * g.dy.sh;
    T* du = (T*)g.du.data + b * g.du.sb + at * g.du.sl + (int64_t)grp * D * g.du.sh;
    T* dz = a.gate ? (T*)g.dz.data + b * g.dz.sb + at * g.dz.sl + (int64_t)grp * D * g.dz.sh : nullptr;
    const Stats s = step_stats<T>(a, u, z, D, live, wave, lane, parts);
    float m0 = 0.0f, m1 = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
        float c0 = 0.0f, c1 = 0.0f;
        if (pass) {
            parts[wave][0][lane] = m0, parts[wave][1][lane] = m1;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kStepWaves; ++i) c0 += parts[i][0][lane], c1 += parts[i][1][lane];
            c0 = a.rms ? 0.0f : c0 / (float)D, c1 /= (float)D;
        }
        for (int k0 = wave * kBlock; k0 < D; k0 += kStepWaves * kBlock) {
            float x[kBlock], e[kBlock], d[kBlock];
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                x[i] = e[i] = d[i] = 0.0f;
                if (live && k0 + i < D) {
                    x[i] = to_f(u[(k0 + i) * a.u.sh]);
                    if (a.gate) e[i] = to_f(z[(k0 + i) * a.z.sh]);
                    d[i] = to_f(dy[(k0 + i) * g.dy.sh]);
                }
            }
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                if (k0 + i >= D) break;
                const int c = grp * D + k0 + i;
                const float w = a.weight ? a.weight[c] : 1.0f, gate = a.gate ? silu_f<kFine<T>>(e[i]) : 1.0f;
                const float n = ((a.gate == SSM_GATE_BEFORE ? x[i] * gate : x[i]) - s.mean) * s.scale;
                const float dp = a.gate == SSM_GATE_AFTER ? d[i] * gate : d[i], dn = dp * w;
                if (pass == 0) {
                    m0 += dn;
                    m1 = fmaf(dn, n, m1);
                    if (g.parts) {
                        const float p = wave_sum(live ? dp * n : 0.0f), q = wave_sum(live ? dp : 0.0f);
                        if (lane == 0) g.parts[block * a.H + c] = p, g.parts[(g.rows + block) * a.H + c] = q;
                    }
                } else if (live) {
                    float o = s.scale * (dn - c0 - n * c1);
                    if (a.gate == SSM_GATE_AFTER)
                        dz[(k0 + i) * g.dz.sh] =
                            from_f<T>(d[i] * fmaf(n, w, a.bias ? a.bias[c] : 0.0f) * silu_slope<T>(e[i]));
                    if (a.gate == SSM_GATE_BEFORE) {
                        dz[(k0 + i) * g.dz.sh] = from_f<T>(o * x[i] * silu_slope<T>(e[i]));
                        o *= gate;
                    }
                    du[(k0 + i) * g.du.sh] = from_f<T>(o);
                }
            }
        }
    }
}

// The parameters' gradients: the rows of partial sums added up in float64, 64 channels
// to a workgroup and sixteen threads to a channel.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const NormGradArgs g) {
    __shared__ double part[16][64];
    const int tid = threadIdx.x, c = tid & 63, k = tid >> 6;
    const int64_t h = (int64_t)blockIdx.x * 64 + c, H = g.f.H;
    for (int which = 0; which < 2; ++which) {
        float* to = which ? g.dbias : g.dweight;
        if (!to) continue;
        double sum = 0.0;
        if (h < H)
            for (int64_t r = k; r < g.rows; r += 16) sum += g.parts[(which * g.rows + r) * H + h];
        part[k][c] = sum;
        __syncthreads();
        if (k == 0 && h < H) {
            for (int i = 1; i < 16; ++i) sum += part[i][c];
            to[h] = (float)sum;
        }
        __syncthreads();
    }
}

// ---- launches ----
// the channels of a group at a step that fit registers; beyond, the other order's kernels serve
constexpr int64_t kMostChannels = 32768, kMostChannelsGrad = 16384;

static bool by_channel(const View3* const* v, int n) {
    for (int i = 0; i < n; ++i)
        if (v[i]->data && v[i]->sh != 1) return false;
    return true;
}
// threads of a step's group
static int norm_lanes(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : D <= 1024 ? 64 : D <= 4096 ? 256 : 1024; }
static int64_t step_blocks(int64_t L) { return (L + 63) / 64; }
// rows of partial sums: the workgroups that go over the steps, times the steps of each
static int64_t norm_rows(int64_t steps, int64_t D, int64_t G) {
    const int64_t R = norm_threads(norm_lanes(D)) / norm_lanes(D);
    int64_t wgs = ((D > 4096 ? 512 : 1024) + G - 1) / G;
    if (wgs * R > steps) wgs = (steps + R - 1) / R;
    return wgs * R;
}
int64_t norm_part_rows(int64_t Bsz, int64_t L, int64_t D, int64_t G) {
    const int64_t a = norm_rows(Bsz * L, D, G), b = Bsz * step_blocks(L);
    return a > b ? a : b;  // either order of the tensors
}
bool norm_fits(int64_t Bsz, int64_t L, int64_t D, int64_t G) {
    const int64_t steps = Bsz * step_blocks(L), most = (int64_t)1 << 32;
    return Bsz * L < most && G < most && Bsz * L < most / G && grid_fits(Bsz * L * G, norm_lanes(D)) && grid_fits(steps * G, kStepThreads);
}

template <class T, int LANES, int V>
static void launch_rows(const NormArgs& a, hipStream_t s) {
    constexpr int R = norm_threads(LANES) / LANES;
    const int64_t rows = a.Bsz * a.L * a.G;
    hipLaunchKernelGGL((norm_rows_kernel<T, LANES, V>), dim3((unsigned)((rows + R - 1) / R)), dim3(norm_threads(LANES)), 0, s,
                       a);
}
template <class T>
static void launch_norm_t(const NormArgs& a, hipStream_t s) {
    const int64_t D = a.H / a.G, blocks = step_blocks(a.L);
    const View3* v[] = {&a.u, &a.z, &a.y};
    if (D > kMostChannels || !by_channel(v, 3))
        hipLaunchKernelGGL((norm_steps_kernel<T>), dim3((unsigned)(a.Bsz * blocks * a.G)), dim3(kStepThreads), 0, s, a, blocks);
    else if (D <= 64) launch_rows<T, 8, 1>(a, s);
    else if (D <= 128) launch_rows<T, 16, 1>(a, s);
    else if (D <= 256) launch_rows<T, 32, 1>(a, s);
    else if (D <= 512) launch_rows<T, 64, 1>(a, s);
    else if (D <= 1024) launch_rows<T, 64, 2>(a, s);
    else if (D <= 2048) launch_rows<T, 256, 1>(a, s);
    else if (D <= 4096) launch_rows<T, 256, 2>(a, s);
    else if (D <= 8192) launch_rows<T, 1024, 1>(a, s);
    else launch_rows<T, 1024, 4>(a, s);
}
hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t s) {
    if (dtype == SSM_F32) launch_norm_t<float>(a, s);
    else if (dtype == SSM_BF16) launch_norm_t<bf16>(a, s);
    else launch_norm_t<f16>(a, s);
    return hipGetLastError();
}

template <class T, int LANES, int V>
static void launch_rows_grad(const NormGradArgs& g, hipStream_t s) {
    constexpr int R = norm_threads(LANES) / LANES;
    hipLaunchKernelGGL((norm_rows_grad_kernel<T, LANES, V>), dim3((unsigned)(g.rows / R * g.f.G)), dim3(norm_threads(LANES)),
                       0, s, g);
}
template <class T>
static void launch_norm_grad_t(NormGradArgs& g, hipStream_t s) {
    const NormArgs& a = g.f;
    const int64_t D = a.H / a.G, blocks = step_blocks(a.L);
    const View3* v[] = {&a.u, &a.z, &g.dy, &g.du, &g.dz};
    if (D > kMostChannelsGrad || !by_channel(v, 5)) {
        g.rows = a.Bsz * blocks;
        hipLaunchKernelGGL((norm_steps_grad_kernel<T>), dim3((unsigned)(a.Bsz * blocks * a.G)), dim3(kStepThreads), 0, s, g,
                           blocks);
        return;
    }
    g.rows = norm_rows(a.Bsz * a.L, D, a.G);
    if (D <= 64) launch_rows_grad<T, 8, 1>(g, s);
    else if (D <= 128) launch_rows_grad<T, 16, 1>(g, s);
    else if (D <= 256) launch_rows_grad<T, 32, 1>(g, s);
    else if (D <= 512) launch_rows_grad<T, 64, 1>(g, s);
    else if (D <= 1024) launch_rows_grad<T, 64, 2>(g, s);
    else if (D <= 2048) launch_rows_grad<T, 256, 1>(g, s);
    else if (D <= 4096) launch_rows_grad<T, 256, 2>(g, s);
    else if (D <= 8192) launch_rows_grad<T, 1024, 1>(g, s);
    else launch_rows_grad<T, 1024, 2>(g, s);
}
hipError_t launch_norm_backward(int dtype, NormGradArgs& g, hipStream_t s) {
    if (dtype == SSM_F32) launch_norm_grad_t<float>(g, s);
    else if (dtype == SSM_BF16) launch_norm_grad_t<bf16>(g, s);
    else launch_norm_grad_t<f16>(g, s);
    if (g.parts) hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((g.f.H + 63) / 64)), dim3(1024), 0, s, g);
    return hipGetLastError();
}

}  // namespace ssm

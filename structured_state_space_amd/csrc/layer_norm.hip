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
// mean first, then the squares about it) and are written once.  Bound by memory: gated, bf16,
// 16384 steps of 2048 channels 38 us, 5.3 TB/s with part of the traffic in the last-level cache.
// `turn` counts the sums of a workgroup: two places in turn need one barrier each.
template <int LANES>
using Parts = float[2][LANES > 64 ? LANES / 64 : 1];
template <int LANES>
__device__ __forceinline__ float group_sum(float v, Parts<LANES>& parts, int& turn) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    if constexpr (LANES > 8) v += dpp<0x140>(v);
    if constexpr (LANES > 16) v += __shfl_xor(v, 16);
    if constexpr (LANES > 32) v += __shfl_xor(v, 32);
    if constexpr (LANES > 64) {
        float* part = parts[turn++ & 1];
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
// the same, left as words as they are in memory (the next step's, on their way)
template <class T>
struct Raw8 {
    u32x4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const void* data, int64_t at, int there) {
        const T* p = (const T*)data + at;
        if (there >= 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const Words<T>*>(p + 16 / sizeof(T) * i)->v;
        } else {
            T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = i < there ? p[i] : from_f<T>(0.0f);
            __builtin_memcpy(w, e, sizeof(e));
        }
    }
    __device__ __forceinline__ void get(float (&r)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) r[i] = __uint_as_float(w[i / 4][i % 4]);
            else r[i] = to_f(__builtin_bit_cast(T, (uint16_t)(w[0][i / 2] >> (16 * (i & 1)))));
        }
    }
};
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
    __shared__ Parts<LANES> parts;
    int turn = 0;
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
    const float mean = a.rms ? 0.0f : group_sum<LANES>(sum, parts, turn) / (float)D;
    float squares = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[v][i] = i < there[v] ? x[v][i] - mean : 0.0f;
            squares = fmaf(x[v][i], x[v][i], squares);
        }
    const float scale = inverse_root(group_sum<LANES>(squares, parts, turn) / (float)D + a.eps);
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
// the forward pass.  Workgroups go over their steps with the same channels in the same lanes, so
// that the parameters' sums stay in registers until the end; each then joins those of its lanes
// and has a row of partial sums.  (A row for each step that a workgroup has at once, 32 of 64
// channels: 16 x 2048 steps took 507 us, most of it the rows' sums.)
template <class T, int LANES, int V>
__global__ __launch_bounds__(norm_threads(LANES)) void norm_rows_grad_kernel(const NormGradArgs g) {
    const NormArgs& a = g.f;
    constexpr int R = norm_threads(LANES) / LANES;
    __shared__ Parts<LANES> parts;
    int turn = 0;
    const int tid = threadIdx.x, D = (int)(a.H / a.G);
    const int grp = (int)(blockIdx.x % a.G);
    const int64_t mine = (int64_t)(blockIdx.x / a.G) * R + tid / LANES, apart = g.rows * R;
    const int first = tid % LANES * 8;
    const int64_t steps = a.Bsz * a.L;
    // Four vectors of everything do not fit the registers: nothing is loaded ahead, and the sums are
    // in LDS, a place for each thread.  (1024 threads with two vectors each had 360 bytes of a
    // thread in memory: 2 x 2048 steps of 16384 channels, bf16, 580 us instead of 237.)
    constexpr bool TIGHT = V == 4;
    __shared__ float kept[TIGHT ? 2 * V * 8 : 1][TIGHT ? LANES : 1];
    float dw[TIGHT ? 1 : V][8], db[TIGHT ? 1 : V][8], w[V][8], s[V][8];
    auto parameters = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = first + v * LANES * 8, there = D - c;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[v][i] = 1.0f, s[v][i] = 0.0f;
            if (a.weight) load8<float>(w[v], a.weight, grp * D + c, there);
            if (a.bias && a.gate == SSM_GATE_AFTER) load8<float>(s[v], a.bias, grp * D + c, there);
        }
    };
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (TIGHT) kept[v * 8 + i][tid] = kept[(V + v) * 8 + i][tid] = 0.0f;
            else dw[v][i] = db[v][i] = 0.0f;
        }
    if (!TIGHT) parameters();
    Raw8<T> un[V], zn[V], dn[V];
    auto load = [&](int64_t r) {
        const int64_t l = r % a.L, b = r / a.L;
        const int64_t u0 = b * a.u.sb + l * a.u.sl + grp * D, z0 = b * a.z.sb + l * a.z.sl + grp * D;
        const int64_t y0 = b * g.dy.sb + l * g.dy.sl + grp * D;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = first + v * LANES * 8, there = D - c;
            un[v].load(a.u.data, u0 + c, there);
            if (a.gate) zn[v].load(a.z.data, z0 + c, there);
            dn[v].load(g.dy.data, y0 + c, there);
        }
    };
    if (!TIGHT && mine < steps) load(mine);
    for (int64_t r = mine; r < steps; r += apart) {
        const int64_t l = r % a.L, b = r / a.L;
        float u[V][8], z[V][8], d[V][8], n[V][8];
        if (TIGHT) load(r);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            un[v].get(u[v]);
            if (a.gate) zn[v].get(z[v]);
            dn[v].get(d[v]);
        }
        if (!TIGHT && r + apart < steps) load(r + apart);
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = first + v * LANES * 8 + i < D;
                n[v][i] = a.gate == SSM_GATE_BEFORE ? (in ? gated<T>(u[v][i], z[v][i], a.gate) : 0.0f) : u[v][i];
                sum += n[v][i];
            }
        const float mean = a.rms ? 0.0f : group_sum<LANES>(sum, parts, turn) / (float)D;
        float squares = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[v][i] = first + v * LANES * 8 + i < D ? n[v][i] - mean : 0.0f;
                squares = fmaf(n[v][i], n[v][i], squares);
            }
        const float scale = inverse_root(group_sum<LANES>(squares, parts, turn) / (float)D + a.eps);
        if (TIGHT) parameters();
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
                if constexpr (TIGHT) {
                    kept[v * 8 + i][tid] += d[v][i] * n[v][i];
                    kept[(V + v) * 8 + i][tid] += d[v][i];
                } else {
                    dw[v][i] = fmaf(d[v][i], n[v][i], dw[v][i]);
                    db[v][i] += d[v][i];
                }
                d[v][i] *= w[v][i];
                m0 += d[v][i];
                m1 = fmaf(d[v][i], n[v][i], m1);
            }
            if (a.gate == SSM_GATE_AFTER && there > 0) store8<T>(dz, g.dz.data, dz0 + c, there);
        }
        const float c0 = a.rms ? 0.0f : group_sum<LANES>(m0, parts, turn) / (float)D;
        const float c1 = group_sum<LANES>(m1, parts, turn) / (float)D;
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
    if (!g.parts) return;
    if constexpr (R > 1) {  // the lanes of the same channels, in a wave and in the others
        constexpr int W = norm_threads(LANES) / 64;
        __shared__ float all[W][LANES * V * 8];
        auto join = [&](auto& x) {
            float* at = all[tid >> 6];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (LANES < 16) x[v][i] += dpp<0x140>(dpp<0x141>(x[v][i]));  // eight lanes on
                    if constexpr (LANES < 32) x[v][i] += __shfl_xor(x[v][i], 16);
                    if constexpr (LANES < 64) x[v][i] += __shfl_xor(x[v][i], 32);
                    if ((tid & 63) < LANES) at[(v * 8 + i) * LANES + (tid & 63)] = x[v][i];
                }
            __syncthreads();
            if (tid < LANES) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int k = 1; k < W; ++k) x[v][i] += all[k][(v * 8 + i) * LANES + tid];
            }
            __syncthreads();
        };
        join(dw), join(db);
        if (tid >= LANES) return;
    }
    const int64_t row = blockIdx.x / a.G;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = first + v * LANES * 8, there = D - c;
        if (there <= 0) continue;
        if constexpr (TIGHT) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[0][i] = kept[v * 8 + i][tid], db[0][i] = kept[(V + v) * 8 + i][tid];
        }
        store8<float>(dw[TIGHT ? 0 : v], g.parts, row * a.H + grp * D + c, there);
        store8<float>(db[TIGHT ? 0 : v], g.parts, (g.rows + row) * a.H + grp * D + c, there);
    }
}

// ---- any other order: 64 steps to a workgroup ----
// A lane has four neighbouring steps, which are one vector where steps are contiguous, and R
// channels: sixteen lanes make a row of 64 steps, 64 rows of lanes share the channels.  The
// numbers stay in registers where they fit (KEEP); else a lane goes over its channels R at a
// time, once for the sums and once for the results.  Means and squares are joined from blocks
// of R, the squares about the joined mean (m2 + m2' + delta^2 n n' / (n + n')).
// (With a step to a lane, 64 channels apart, loads were four bytes wide and a channel's sum
// over the steps went through all lanes: 16 x 512 x 3000, float32: 72 us, gradients 178.)
constexpr int kSteps = 64;
constexpr int kStepThreads = 1024;
constexpr int kStepWaves = kStepThreads / 64;
constexpr int kStepParts = kStepWaves * 4;

// four steps of a channel, as words
template <class T>
struct Four {
    uint32_t w[sizeof(T)];
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else return to_f(__builtin_bit_cast(T, (uint16_t)(w[j / 2] >> (16 * (j & 1)))));
    }
};
// One tensor at a lane's four steps of a group's channels.  VEC: steps are contiguous and a
// group within 2^32 bytes: a base for the whole workgroup and 32 bits a lane.  (With 64-bit
// addresses per lane and both ways in one kernel the numbers did not fit the registers.)
template <class T, bool VEC>
struct Column {
    const char* base;
    uint32_t sh, sl, off;  // bytes
    int there;             // steps that exist (without VEC; see steps_of)
    __device__ __forceinline__ Column(const View3& v, int64_t b, int64_t block, int64_t c, int step, int steps)
        : base((const char*)v.data + (b * v.sb + (block - (VEC ? 4 : 0)) * v.sl + c * v.sh) * (int64_t)sizeof(T)),
          sh((uint32_t)v.sh * (uint32_t)sizeof(T)), sl((uint32_t)v.sl * (uint32_t)sizeof(T)),
          off((uint32_t)(step + (VEC ? 4 : 0)) * sl), there(steps) {}
    __device__ __forceinline__ Four<T> load(int c) const {
        Four<T> f = {};
        if constexpr (VEC) {
            struct __attribute__((packed, aligned(sizeof(T)))) Packed { Four<T> f; };
            f = reinterpret_cast<const Packed*>(base + (uint32_t)((uint32_t)c * sh + off))->f;
        } else {
            const char* at = base + (int64_t)c * sh + off;
            T e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = j < there ? *reinterpret_cast<const T*>(at + (int64_t)j * sl) : from_f<T>(0.0f);
            __builtin_memcpy(&f, e, sizeof(f));
        }
        return f;
    }
    __device__ __forceinline__ void store(int c, const float (&r)[4]) const {
        if constexpr (VEC) {
            Vec4<T> w;
#pragma unroll
            for (int j = 0; j < 4; ++j) w.v[j] = from_f<T>(r[j]);
            *reinterpret_cast<Vec4<T>*>((char*)base + (uint32_t)((uint32_t)c * sh + off)) = w;
        } else {
            char* at = (char*)base + (int64_t)c * sh + off;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < there) *reinterpret_cast<T*>(at + (int64_t)j * sl) = from_f<T>(r[j]);
        }
    }
    template <int R>
    __device__ __forceinline__ void load_all(Four<T> (&r)[R], int c0, int D) const {  // channels behind the last read it again
#pragma unroll
        for (int i = 0; i < R; ++i) r[i] = load(min(c0 + i, D - 1));
    }
};
// A lane's first step within the workgroup's block, of which L - block * kSteps are left.  VEC: a
// vector that would pass the last step is moved back to end with it; of its steps those from
// `fresh` on are the lane's own, the others another lane's, which computes and stores the same.
// Else `there` of the steps exist.
template <bool VEC>
__device__ __forceinline__ void steps_of(int q, int64_t left, int& step, int& there, int& fresh) {
    const int n = (int)min((int64_t)kSteps, left);
    step = 4 * q;
    there = max(0, min(4, n - step));
    fresh = 0;
    if (VEC) {
        const int back = min(step, n - 4);  // (may lie before the block: L is at least 4)
        fresh = min(4, step - back);
        step = back;
    } else {
        step = min(step, n - 1);
    }
}
template <class T, int R>
__device__ __forceinline__ void fresh(Four<T> (&f)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < (int)sizeof(T); ++j) asm volatile("" : "+v"(f[i].w[j]));
}
struct Running {
    float count = 0.0f, mean = 0.0f, m2 = 0.0f;
    __device__ __forceinline__ void join(float n, float mu, float q) {
        const float all = count + n, share = all > 0.0f ? n * __builtin_amdgcn_rcpf(all) : 0.0f, delta = mu - mean;
        mean = fmaf(delta, share, mean);
        m2 += q + delta * delta * count * share;
        count = all;
    }
};
template <class T, int R>
__device__ __forceinline__ void join_block(Running (&s)[4], const NormArgs& a, const Four<T> (&u)[R], const Four<T> (&z)[R], int c0,
                                           int D) {
    const int n = min(R, D - c0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x[R], sum = 0.0f, squares = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            x[i] = u[i].get(j);
            if (a.gate == SSM_GATE_BEFORE) x[i] = gated<T>(x[i], z[i].get(j), a.gate);
            sum += i < n ? x[i] : 0.0f;
        }
        const float mean = a.rms ? 0.0f : sum / (float)n;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float d = i < n ? x[i] - mean : 0.0f;
            squares = fmaf(d, d, squares);
        }
        s[j].join((float)n, mean, squares);
    }
}
// Sums over the workgroup go by the rows of a wave's lanes, then by LDS, where a wave has four
// steps and a lane for each other wave.
struct StepParts {
    float part[3][kStepWaves][kSteps];
    float all[2][kSteps];
};
__device__ __forceinline__ void join_all(Running (&s)[4], Stats (&stats)[4], StepParts& sh, int D, float eps, int lane, int wave) {
    const int q = lane & 15;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int d = 16; d < 64; d <<= 1) {
            const float n = __shfl_xor(s[j].count, d), m = __shfl_xor(s[j].mean, d), v = __shfl_xor(s[j].m2, d);
            s[j].join(n, m, v);
        }
    }
    if (lane < 16) {
        *reinterpret_cast<f32x4*>(&sh.part[0][wave][4 * q]) = f32x4{s[0].count, s[1].count, s[2].count, s[3].count};
        *reinterpret_cast<f32x4*>(&sh.part[1][wave][4 * q]) = f32x4{s[0].mean, s[1].mean, s[2].mean, s[3].mean};
        *reinterpret_cast<f32x4*>(&sh.part[2][wave][4 * q]) = f32x4{s[0].m2, s[1].m2, s[2].m2, s[3].m2};
    }
    __syncthreads();
    const int step = 4 * wave + (lane >> 4);
    Running r;
    r.count = sh.part[0][q][step], r.mean = sh.part[1][q][step], r.m2 = sh.part[2][q][step];
    r.join(dpp<0xB1>(r.count), dpp<0xB1>(r.mean), dpp<0xB1>(r.m2));
    r.join(dpp<0x4E>(r.count), dpp<0x4E>(r.mean), dpp<0x4E>(r.m2));
    r.join(dpp<0x141>(r.count), dpp<0x141>(r.mean), dpp<0x141>(r.m2));
    r.join(dpp<0x140>(r.count), dpp<0x140>(r.mean), dpp<0x140>(r.m2));
    if (q == 0) sh.all[0][step] = r.mean, sh.all[1][step] = inverse_root(r.m2 / (float)D + eps);
    __syncthreads();
    const f32x4 m = *reinterpret_cast<const f32x4*>(&sh.all[0][4 * q]), v = *reinterpret_cast<const f32x4*>(&sh.all[1][4 * q]);
#pragma unroll
    for (int j = 0; j < 4; ++j) stats[j] = {m[j], v[j]};
}
// two sums; `sh` has been read since the last call
__device__ __forceinline__ void sum_all(float (&x)[4], float (&y)[4], StepParts& sh, int lane, int wave) {
    const int q = lane & 15;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = across_rows(x[j]), y[j] = across_rows(y[j]);
    if (lane < 16) {
        *reinterpret_cast<f32x4*>(&sh.part[0][wave][4 * q]) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4*>(&sh.part[1][wave][4 * q]) = f32x4{y[0], y[1], y[2], y[3]};
    }
    __syncthreads();
    const int step = 4 * wave + (lane >> 4);
    const float p = row_sum(sh.part[0][q][step]), r = row_sum(sh.part[1][q][step]);
    if (q == 0) sh.all[0][step] = p, sh.all[1][step] = r;
    __syncthreads();
    const f32x4 m = *reinterpret_cast<const f32x4*>(&sh.all[0][4 * q]), v = *reinterpret_cast<const f32x4*>(&sh.all[1][4 * q]);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = m[j], y[j] = v[j];
}
// the channels' parameters, at clamped places as the tensors
template <int R>
__device__ __forceinline__ void load_parameters(float (&w)[R], const float* p, float none, int c0, int D) {
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = p ? p[min(c0 + i, D - 1)] : none;
}

template <class T, int R, bool KEEP, bool GATED, bool VEC>
__global__ __launch_bounds__(kStepThreads) void norm_steps_kernel(const NormArgs a, int64_t blocks) {
    __shared__ __attribute__((aligned(16))) StepParts parts;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = threadIdx.x >> 4;
    // neighbouring blocks of steps share cache lines: on one die (46 us instead of 50 at 16 x 512 x 3000)
    const int64_t bid = by_die(blockIdx.x, gridDim.x);
    const int D = (int)(a.H / a.G), grp = (int)(bid / blocks % a.G);
    const int64_t block = bid % blocks * kSteps, b = bid / blocks / a.G, first = (int64_t)grp * D;
    int step, there, own;
    steps_of<VEC>(lane & 15, a.L - block, step, there, own);
    const Column<T, VEC> uc(a.u, b, block, first, step, there), zc(GATED ? a.z : a.u, b, block, first, step, there);
    const Column<T, VEC> yc(a.y, b, block, first, step, there);
    const float *weight = a.weight ? a.weight + first : nullptr, *bias = a.bias ? a.bias + first : nullptr;
    Four<T> u[R], z[R];
    float w[R], shift[R];
    Running run[4];
    Stats s[4];
    for (int c0 = part * R; c0 < D; c0 += KEEP ? D : kStepParts * R) {
        uc.load_all(u, c0, D);
        if (GATED) zc.load_all(z, c0, D);
        join_block<T, R>(run, a, u, GATED ? z : u, c0, D);
    }
    join_all(run, s, parts, D, a.eps, lane, wave);
    for (int c0 = part * R; c0 < D; c0 += KEEP ? D : kStepParts * R) {
        if (!KEEP) {
            uc.load_all(u, c0, D);
            if (GATED) zc.load_all(z, c0, D);
        }
        load_parameters(w, weight, 1.0f, c0, D), load_parameters(shift, bias, 0.0f, c0, D);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = u[i].get(j), e = GATED ? silu_f<kFine<T>>(z[i].get(j)) : 1.0f;
                y[j] = fmaf(((GATED && a.gate == SSM_GATE_BEFORE ? x * e : x) - s[j].mean) * s[j].scale, w[i], shift[i]);
                if (GATED && a.gate == SSM_GATE_AFTER) y[j] *= e;
            }
            if (c0 + i < D) yc.store(c0 + i, y);
        }
    }
}

// Gradients: a channel's sums over the steps are sums over the lanes of a row, added up in the
// workgroup's row of partial sums over the blocks of steps that it takes.
template <class T, int R, bool KEEP, bool GATED, bool VEC>
__global__ __launch_bounds__(kStepThreads) void norm_steps_grad_kernel(const NormGradArgs g, int64_t blocks) {
    const NormArgs& a = g.f;
    __shared__ __attribute__((aligned(16))) StepParts parts;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = threadIdx.x >> 4, q = lane & 15;
    const int64_t bid = by_die(blockIdx.x, gridDim.x);
    const int D = (int)(a.H / a.G), grp = (int)(bid / g.rows);
    const int64_t first = (int64_t)grp * D, mine = bid % g.rows;
    float* sums = g.parts ? g.parts + mine * a.H + first : nullptr;
    const float *weight = a.weight ? a.weight + first : nullptr, *bias = a.bias ? a.bias + first : nullptr;
    for (int64_t block = mine; block < a.Bsz * blocks; block += g.rows) {
        const int64_t at = block % blocks * kSteps, b = block / blocks;
        const bool again = block != mine;
        int step, there, own;
        steps_of<VEC>(q, a.L - at, step, there, own);
        if (VEC) there = 4;
        const Column<T, VEC> uc(a.u, b, at, first, step, there), zc(GATED ? a.z : a.u, b, at, first, step, there);
        const Column<T, VEC> dyc(g.dy, b, at, first, step, there), duc(g.du, b, at, first, step, there);
        const Column<T, VEC> dzc(GATED ? g.dz : g.du, b, at, first, step, there);
        Four<T> u[R], z[R], dy[R];
        float w[R], shift[R];
        Running run[4];
        Stats s[4];
        auto load = [&](int c0) {
            uc.load_all(u, c0, D);
            if (GATED) zc.load_all(z, c0, D);
            dyc.load_all(dy, c0, D);
            load_parameters(w, weight, 1.0f, c0, D);
            if (GATED) load_parameters(shift, bias, 0.0f, c0, D);
        };
        // the normed number, and the gradient of the result in front of a gate
        auto parts_of = [&](int i, int j, float& n, float& d, float& gate) {
            const float x = u[i].get(j);
            gate = GATED ? silu_f<kFine<T>>(z[i].get(j)) : 1.0f;
            n = ((GATED && a.gate == SSM_GATE_BEFORE ? x * gate : x) - s[j].mean) * s[j].scale;
            d = GATED && a.gate == SSM_GATE_AFTER ? dy[i].get(j) * gate : dy[i].get(j);
        };
        for (int c0 = part * R; c0 < D; c0 += KEEP ? D : kStepParts * R) {
            if (KEEP) load(c0);
            else {
                uc.load_all(u, c0, D);
                if (GATED) zc.load_all(z, c0, D);
            }
            join_block<T, R>(run, a, u, GATED ? z : u, c0, D);
        }
        join_all(run, s, parts, D, a.eps, lane, wave);
        if (KEEP) fresh(u);
        if (KEEP && GATED) fresh(z);
        float m0[4] = {0, 0, 0, 0}, m1[4] = {0, 0, 0, 0};
        for (int c0 = part * R; c0 < D; c0 += KEEP ? D : kStepParts * R) {
            if (!KEEP) load(c0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float in = c0 + i < D ? w[i] : 0.0f;
                float p = 0.0f, r = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float n, d, gate;
                    parts_of(i, j, n, d, gate);
                    m0[j] = fmaf(d, in, m0[j]);
                    m1[j] = fmaf(d * in, n, m1[j]);
                    p += j >= own && j < there ? d * n : 0.0f, r += j >= own && j < there ? d : 0.0f;
                }
                if (sums) {
                    p = row_sum(p), r = row_sum(r);
                    if (q == 0 && c0 + i < D) {
                        float* to = sums + c0 + i;
                        if (again) p += to[0], r += to[g.rows * a.H];
                        to[0] = p, to[g.rows * a.H] = r;
                    }
                }
            }
        }
        sum_all(m0, m1, parts, lane, wave);
#pragma unroll
        for (int j = 0; j < 4; ++j) m0[j] = a.rms ? 0.0f : m0[j] / (float)D, m1[j] /= (float)D;
        // what was worked out above is worked out again: kept, it would not fit the registers
        fresh(u), fresh(dy);
        if (GATED) fresh(z);
        for (int c0 = part * R; c0 < D; c0 += KEEP ? D : kStepParts * R) {
            if (!KEEP) load(c0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float du[4], dz[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float n, d, gate;
                    parts_of(i, j, n, d, gate);
                    du[j] = s[j].scale * (d * w[i] - m0[j] - n * m1[j]);
                    if (GATED && a.gate == SSM_GATE_AFTER) dz[j] = dy[i].get(j) * fmaf(n, w[i], shift[i]) * silu_slope<T>(z[i].get(j));
                    if (GATED && a.gate == SSM_GATE_BEFORE) {
                        dz[j] = du[j] * u[i].get(j) * silu_slope<T>(z[i].get(j));
                        du[j] *= gate;
                    }
                }
                if (c0 + i < D) {
                    duc.store(c0 + i, du);
                    if (GATED) dzc.store(c0 + i, dz);
                }
            }
        }
    }
}

// The parameters' gradients: the rows of partial sums added up in float64, sixteen channels
// to a workgroup at a time and sixteen threads to a channel, eight rows under way.
__global__ __launch_bounds__(256) void norm_sums_kernel(const NormGradArgs g) {
    __shared__ double part[16][16];
    const int tid = threadIdx.x, c = tid & 15, k = tid >> 4;
    const int64_t H = g.f.H, blocks = (H + 15) / 16;
    for (int64_t unit = blockIdx.x; unit < 2 * blocks; unit += gridDim.x) {
        const int64_t h = unit % blocks * 16 + c;
        const int which = (int)(unit / blocks);
        float* to = which ? g.dbias : g.dweight;
        if (!to) continue;
        double sum = 0.0;
        if (h < H)
            for (int64_t r = k; r < g.rows; r += 16 * 8) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = r + 16 * i < g.rows ? g.parts[(which * g.rows + r + 16 * i) * H + h] : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += v[i];
            }
        __syncthreads();  // the last channels' sums have been read
        part[k][c] = sum;
        __syncthreads();
        if (k == 0 && h < H) {
            for (int i = 1; i < 16; ++i) sum += part[i][c];
            to[h] = (float)sum;
        }
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
// Threads of a step's group, with one or two vectors each: 2048 channels, gated, bf16, 8192 steps, 25 us;
// four vectors each, in a quarter of the threads, 34.
static int norm_lanes(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : D <= 1024 ? 64 : D <= 4096 ? 256 : 1024; }
static int norm_grad_lanes(int64_t D) { return D > 4096 ? 512 : norm_lanes(D); }
static int64_t step_blocks(int64_t L) { return (L + kSteps - 1) / kSteps; }
// Rows of partial sums: the workgroups that go over a group's steps, two to a compute unit (one of
// 512 or 1024 threads).  Gated, bf16: 8192 steps of 4096 channels 93 us, with half as many 130;
// 32768 of 512 55 us and of 64 24 us, with twice as many 63 and 31.
static int64_t norm_rows(int64_t steps, int64_t D, int64_t G) {
    const int64_t R = norm_threads(norm_grad_lanes(D)) / norm_grad_lanes(D);
    const int64_t wgs = ((D > 4096 ? 256 : 512) + G - 1) / G, all = (steps + R - 1) / R;
    return wgs < all ? wgs : all;
}
// Of the other order's, one to a compute unit: 16 x 512 x 3000, float32, 113 us, half as many 156, twice 132.
static int64_t norm_step_rows(int64_t Bsz, int64_t L, int64_t G) {
    const int64_t all = Bsz * step_blocks(L), most = (256 + G - 1) / G;
    return all < most ? all : most;
}
int64_t norm_part_rows(int64_t Bsz, int64_t L, int64_t D, int64_t G) {
    const int64_t a = norm_rows(Bsz * L, D, G), b = norm_step_rows(Bsz, L, G);
    return a > b ? a : b;  // either order of the tensors
}
// The two orders' grids, forwards and backwards; a call is refused by its own order's alone.
static bool rows_fit(int64_t Bsz, int64_t L, int64_t D, int64_t G, bool grad) {
    const int lanes = (int)(grad ? norm_grad_lanes(D) : norm_lanes(D)), threads = norm_threads(lanes), R = threads / lanes;
    if (Bsz * L >= ((int64_t)1 << 40) / G) return false;
    return grid_fits(grad ? norm_rows(Bsz * L, D, G) * G : (Bsz * L * G + R - 1) / R, threads);
}
static bool steps_fit(int64_t Bsz, int64_t L, int64_t G, bool grad) {
    if (Bsz * step_blocks(L) >= ((int64_t)1 << 40) / G) return false;
    return grid_fits((grad ? norm_step_rows(Bsz, L, G) : Bsz * step_blocks(L)) * G, kStepThreads);
}
static bool rows_order(const NormArgs& a) {
    const View3* v[] = {&a.u, &a.z, &a.y};
    return a.H / a.G <= kMostChannels && by_channel(v, 3);
}
static bool rows_order(const NormGradArgs& g) {
    const View3* v[] = {&g.f.u, &g.f.z, &g.dy, &g.du, &g.dz};
    return g.f.H / g.f.G <= kMostChannelsGrad && by_channel(v, 5);
}
bool norm_fits(const NormArgs& a) {
    return rows_order(a) ? rows_fit(a.Bsz, a.L, a.H / a.G, a.G, false) : steps_fit(a.Bsz, a.L, a.G, false);
}
bool norm_fits(const NormGradArgs& g) {
    const NormArgs& a = g.f;
    return rows_order(g) ? rows_fit(a.Bsz, a.L, a.H / a.G, a.G, true) : steps_fit(a.Bsz, a.L, a.G, true);
}
bool norm_grad_may_fit(int64_t Bsz, int64_t L, int64_t D, int64_t G) {
    return (D <= kMostChannelsGrad && rows_fit(Bsz, L, D, G, true)) || steps_fit(Bsz, L, G, true);
}

template <class T, int LANES, int V>
static void launch_rows(const NormArgs& a, hipStream_t s) {
    constexpr int R = norm_threads(LANES) / LANES;
    const int64_t rows = a.Bsz * a.L * a.G;
    hipLaunchKernelGGL((norm_rows_kernel<T, LANES, V>), dim3((unsigned)((rows + R - 1) / R)), dim3(norm_threads(LANES)), 0, s,
                       a);
}
// Channels of a lane: few where the group has few, more in registers while they fit.  float32, 16 x 3000
// steps: 128 channels 28 us and 512 46 us, read twice instead 30 and 53.  Gradients keep 128 channels
// alone: with 512, or the norm's input of them, registers went to memory (16 x 512 x 3000, dy read twice
// 111 us instead of 113, but 256 channels 72 instead of 64).  Beyond, u is read three times and dy twice:
// 510 MB where 197 would do.  LDS, of which a workgroup has 14 KB of 160, is not used for them.
template <class T, bool GATED, bool VEC>
static void launch_steps(const NormArgs& a, int64_t blocks, hipStream_t s) {
    const int64_t D = a.H / a.G;
    const dim3 grid((unsigned)(a.Bsz * blocks * a.G)), wg(kStepThreads);
    if constexpr (!VEC) hipLaunchKernelGGL((norm_steps_kernel<T, 2, false, GATED, VEC>), grid, wg, 0, s, a, blocks);
    else if (D <= 128) hipLaunchKernelGGL((norm_steps_kernel<T, 2, true, GATED, VEC>), grid, wg, 0, s, a, blocks);
    else if (D <= 512) hipLaunchKernelGGL((norm_steps_kernel<T, 8, true, GATED, VEC>), grid, wg, 0, s, a, blocks);
    else hipLaunchKernelGGL((norm_steps_kernel<T, 8, false, GATED, VEC>), grid, wg, 0, s, a, blocks);
}
template <class T, bool GATED, bool VEC>
static void launch_steps_grad(const NormGradArgs& g, int64_t blocks, hipStream_t s) {
    constexpr int R = GATED && sizeof(T) == 4 ? 2 : 4;
    const int64_t D = g.f.H / g.f.G;
    const dim3 grid((unsigned)(g.rows * g.f.G)), wg(kStepThreads);
    if constexpr (!VEC) hipLaunchKernelGGL((norm_steps_grad_kernel<T, GATED ? 1 : 2, false, GATED, VEC>), grid, wg, 0, s, g, blocks);
    else if (D <= 128) hipLaunchKernelGGL((norm_steps_grad_kernel<T, 2, true, GATED, VEC>), grid, wg, 0, s, g, blocks);
    else hipLaunchKernelGGL((norm_steps_grad_kernel<T, R, false, GATED, VEC>), grid, wg, 0, s, g, blocks);
}
// steps contiguous everywhere, and a group's channels within 32 bits of each other
static bool by_step(const View3* const* v, int n, int64_t D, int64_t L) {
    for (int i = 0; i < n; ++i)
        if (v[i]->data && (v[i]->sl != 1 || v[i]->sh >= ((int64_t)1 << 29) / D)) return false;
    return L >= 4;
}
template <class T>
static void launch_norm_t(const NormArgs& a, hipStream_t s) {
    const int64_t D = a.H / a.G, blocks = step_blocks(a.L);
    const View3* v[] = {&a.u, &a.z, &a.y};
    if (!rows_order(a)) {
        if (by_step(v, 3, D, a.L)) a.gate ? launch_steps<T, true, true>(a, blocks, s) : launch_steps<T, false, true>(a, blocks, s);
        else a.gate ? launch_steps<T, true, false>(a, blocks, s) : launch_steps<T, false, false>(a, blocks, s);
    } else if (D <= 64) launch_rows<T, 8, 1>(a, s);
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
    hipLaunchKernelGGL((norm_rows_grad_kernel<T, LANES, V>), dim3((unsigned)(g.rows * g.f.G)), dim3(norm_threads(LANES)), 0, s, g);
}
template <class T>
static void launch_norm_grad_t(NormGradArgs& g, hipStream_t s) {
    const NormArgs& a = g.f;
    const int64_t D = a.H / a.G, blocks = step_blocks(a.L);
    const View3* v[] = {&a.u, &a.z, &g.dy, &g.du, &g.dz};
    if (!rows_order(g)) {
        g.rows = norm_step_rows(a.Bsz, a.L, a.G);
        if (by_step(v, 5, D, a.L))
            a.gate ? launch_steps_grad<T, true, true>(g, blocks, s) : launch_steps_grad<T, false, true>(g, blocks, s);
        else a.gate ? launch_steps_grad<T, true, false>(g, blocks, s) : launch_steps_grad<T, false, false>(g, blocks, s);
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
    else if (D <= 8192) launch_rows_grad<T, 512, 2>(g, s);
    else launch_rows_grad<T, 512, 4>(g, s);
}
hipError_t launch_norm_backward(int dtype, NormGradArgs& g, hipStream_t s) {
    if (dtype == SSM_F32) launch_norm_grad_t<float>(g, s);
    else if (dtype == SSM_BF16) launch_norm_grad_t<bf16>(g, s);
    else launch_norm_grad_t<f16>(g, s);
    if (g.parts) {  // (a workgroup has several units of channels only where one each would pass a launch's 2^32 threads)
        const int64_t units = (g.f.H + 15) / 16 * 2, most = (int64_t)1 << 23;
        hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)(units < most ? units : most)), dim3(256), 0, s, g);
    }
    return hipGetLastError();
}

}  // namespace ssm

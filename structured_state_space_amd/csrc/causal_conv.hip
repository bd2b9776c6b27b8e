// Short causal convolution per channel, forward and backward:
//   pre_t = bias + sum_k w[k] u_{t-W+1+k},  y_t = pre_t or silu(pre_t)
// with the W - 1 inputs before a sequence's first step taken from its state
// (zero without one), and the state after its last step handed on.
//
// Both directions read and write each element once and are bound by HBM; the
// arithmetic per element is 2 W operations and one exponential (backward 6 W and one).
// bf16, width 4: 4096 channels x 16384 steps 46 us, 5.8 TB/s (part of it from the
// last-level cache; a large copy reaches 4.8); gradients of 4 x 4096 x 2048, 45 us and 4
// for the sums, 4.1 TB/s; by rows, float32, 16 x 512 x 3000, width 3, 70 us and 5,
// 3.9 TB/s.  A small call waits for its few loads: 1536 channels x 5096 packed steps,
// f16, 13 us.
//   tokens  channels contiguous: a thread holds 16 bytes of channels (backward two
//           channels) and walks up to kMaxWalk steps with the W - 1 last inputs in
//           registers; 64 lanes read 1 KB of one step.  Any other strides take one channel.
//   rows    steps contiguous: a thread holds 8 steps of one channel and reads the
//           steps around them again (an L1 hit).
// Backward: dpre_t = dy_t silu'(pre_t) is recomputed, du_t sums W of them, so a
// thread reads W - 1 steps past its own.  The weights' gradients are summed per
// workgroup in a fixed order, written as one row of partial sums per workgroup
// and added up in float64 by a second launch, so a repeated call gives the same bits.
#include "selective.hpp"

namespace ssm {

namespace {

constexpr int kMaxWalk = 64;  // steps a thread walks at most ("tokens"); see geometry()
constexpr int kAhead = 8;     // of them loaded together

template <class T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) VecN {
    T v[V];
};

struct Geometry {
    int Q;        // steps of an item
    int cx;       // threads along the channels (tokens) or along the steps (rows); 256 / cx along the other
    int walk;     // steps a thread walks (tokens)
    int blocks;   // channel blocks
};

template <bool FINE>
__device__ __forceinline__ float silu_slope(float v) {
    const float p = sigmoid_f<FINE>(v);
    return p * fmaf(v, 1.0f - p, 1.0f);
}

// V channels of one step; the last channel block may hold fewer
template <class T, int V>
__device__ __forceinline__ void load_v(float (&r)[V], const T* p, int64_t sh, int n) {
    if (V > 1 && n == V) {
        const VecN<T, V> w = *reinterpret_cast<const VecN<T, V>*>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = to_f(w.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = i < n ? to_f(p[i * sh]) : 0.0f;
    }
}
template <class T, int V>
__device__ __forceinline__ void store_v(const float (&r)[V], T* p, int64_t sh, int n) {
    if (V > 1 && n == V) {
        VecN<T, V> w;
#pragma unroll
        for (int i = 0; i < V; ++i) w.v[i] = from_f<T>(r[i]);
        *reinterpret_cast<VecN<T, V>*>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i * sh] = from_f<T>(r[i]);
    }
}

// the first n of N consecutive elements
template <class T, int N>
__device__ __forceinline__ void load_line(VecN<T, N>& r, const T* p, int n) {
    if (n == N) {
        r = *reinterpret_cast<const VecN<T, N>*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) r.v[i] = p[i];
    }
}
template <class T, int N>
__device__ __forceinline__ void store_line(T* p, const VecN<T, N>& r, int n) {
    if (n == N) {
        *reinterpret_cast<VecN<T, N>*>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = r.v[i];
    }
}

// V channels' weights and biases
template <int W, int V>
__device__ __forceinline__ void load_weights(float (&w)[W][V], float (&b)[V], const float* weight, const float* bias,
                                             int64_t h, int n) {
    if (n == V) {
        const VecN<float, W * V> x = *reinterpret_cast<const VecN<float, W * V>*>(weight + h * W);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = x.v[i * W + k];
        VecN<float, V> y = {};
        if (bias) y = *reinterpret_cast<const VecN<float, V>*>(bias + h);
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = y.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b[i] = bias && i < n ? bias[h + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = i < n ? weight[(h + i) * W + k] : 0.0f;
        }
    }
}

// input `back` steps before the sequence's step 0 (back >= 1), from its state
template <class T, int W>
__device__ __forceinline__ float old_input(const T* state, int64_t row, int64_t H, int h, int back) {
    return state ? to_f(state[(row * H + h) * (W - 1) + (W - 1 - back)]) : 0.0f;
}

// the state after the sequence: its last W - 1 inputs, from u where it has
// them and from the state before it where it is shorter (read before anything
// is written: state_out may be state_in)
template <class T, int W>
__device__ __forceinline__ void hand_on(const ConvArgs& a, const Item& it, int h) {
    if constexpr (W > 1) {
        if (!a.state_out) return;
        const int len = it.end - it.beg;
        T next[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = len - (W - 1) + j;
            if (t >= 0)
                next[j] = ((const T*)a.u.data)[it.row * a.u.sb + h * a.u.sh + (it.beg + t) * a.u.sl];
            else
                next[j] = a.state_in ? ((const T*)a.state_in)[(it.state * a.H + h) * (W - 1) + (W - 1 + t)]
                                     : from_f<T>(0.0f);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) ((T*)a.state_out)[(it.state * a.H + h) * (W - 1) + j] = next[j];
    }
}

template <class T, int W, int V>
__global__ __launch_bounds__(256) void conv_tokens_kernel(ConvArgs a, Geometry geo) {
    const int cb = blockIdx.x % geo.blocks;
    Item it;
    if (!find_item(a.q, blockIdx.x / geo.blocks, geo.Q, it) || it.state < 0) return;
    const int cx = threadIdx.x & (geo.cx - 1), seg = threadIdx.x / geo.cx;
    const int64_t h = ((int64_t)cb * geo.cx + cx) * V;
    if (h >= a.H) return;
    const int n = (int)min((int64_t)V, a.H - h);
    const int64_t first = (int64_t)it.beg + (int64_t)it.c * geo.Q + seg * geo.walk;  // this thread's steps
    const int64_t last = min((int64_t)it.end, first + geo.walk);

    float w[W][V], b[V], past[W > 1 ? W - 1 : 1][V] = {};
    load_weights<W, V>(w, b, a.weight, a.bias, h, n);
    const T* u = (const T*)a.u.data + it.row * a.u.sb + h * a.u.sh;
    T* y = (T*)a.y.data + it.row * a.y.sb + h * a.y.sh;
    // past[k]: the input W - 1 - k steps before `first`; a walk is longer than W - 1
    // steps, so it is in u for every thread but the sequence's first
    if constexpr (W > 1) {
        if (it.c == 0 && seg == 0) {
            VecN<T, V*(W - 1)> old, next;
            const int64_t at = (it.state * a.H + h) * (W - 1);
#pragma unroll
            for (int i = 0; i < V * (W - 1); ++i) old.v[i] = from_f<T>(0.0f);
            if (a.state_in) load_line<T, V*(W - 1)>(old, (const T*)a.state_in + at, n * (W - 1));
#pragma unroll
            for (int i = 0; i < V * (W - 1); ++i) past[i % (W - 1)][i / (W - 1)] = to_f(old.v[i]);
            if (a.state_out) {  // (read above: it may be state_in)
                const int len = it.end - it.beg;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const int t = len - (W - 1) + j;
                    if (t >= 0) {
                        const T* from = u + (it.beg + t) * a.u.sl;
                        if (V > 1 && n == V) {
                            const VecN<T, V> x = *reinterpret_cast<const VecN<T, V>*>(from);
#pragma unroll
                            for (int i = 0; i < V; ++i) next.v[i * (W - 1) + j] = x.v[i];
                        } else {
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                next.v[i * (W - 1) + j] = i < n ? from[i * a.u.sh] : from_f<T>(0.0f);
                        }
                    } else {  // t + W - 1 = len + j
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            next.v[i * (W - 1) + j] = old.v[i * (W - 1)];
#pragma unroll
                            for (int k = 1; k < W - 1; ++k)
                                if (t + W - 1 == k) next.v[i * (W - 1) + j] = old.v[i * (W - 1) + k];
                        }
                    }
                }
                store_line<T, V*(W - 1)>((T*)a.state_out + at, next, n * (W - 1));
            }
        } else if (first < last) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                load_v<T, V>(past[k], u + (first - (W - 1) + k) * a.u.sl, a.u.sh, n);
        }
    }
    auto step = [&](const float (&x)[V], float (&o)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float acc = b[i];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) acc = fmaf(w[k][i], past[k][i], acc);
            o[i] = fmaf(w[W - 1][i], x[i], acc);
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) past[k][i] = past[k + 1][i];
            if (W > 1) past[W > 1 ? W - 2 : 0][i] = x[i];
        }
        if (a.silu) {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = silu_f<kFine<T>>(o[i]);
        }
    };
    int64_t t = first;
    if (V > 1 && n == V) {
        const T* from = u + first * a.u.sl;
        T* to = y + first * a.y.sl;
        for (; t + kAhead <= last; t += kAhead) {
            VecN<T, V> raw[kAhead];
#pragma unroll
            for (int s = 0; s < kAhead; ++s, from += a.u.sl) raw[s] = *reinterpret_cast<const VecN<T, V>*>(from);
#pragma unroll
            for (int s = 0; s < kAhead; ++s, to += a.y.sl) {
                float x[V], o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = to_f(raw[s].v[i]);
                step(x, o);
                VecN<T, V> out;
#pragma unroll
                for (int i = 0; i < V; ++i) out.v[i] = from_f<T>(o[i]);
                *reinterpret_cast<VecN<T, V>*>(to) = out;
            }
        }
    }
    for (; t < last; ++t) {
        float x[V], o[V];
        load_v<T, V>(x, u + t * a.u.sl, a.u.sh, n);
        step(x, o);
        store_v<T, V>(o, y + t * a.y.sl, a.y.sh, n);
    }
}

// steps t - 4 .. t + 7 of a row as 12 floats; outside [beg, end): before it from
// `state` (nullable), behind it 0
template <class T, int W>
__device__ __forceinline__ void row_before(float (&r)[4], const T* p, int64_t t, const Item& it, const T* state,
                                           int64_t H, int h) {
    if (t - 4 >= it.beg) {
        const Vec4<T> v = *reinterpret_cast<const Vec4<T>*>(p + t - 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = to_f(v.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = t - 4 + i;
            const int back = (int)(it.beg - at);
            r[i] = at >= it.beg ? to_f(p[at]) : back < W ? old_input<T, W>(state, it.state, H, h, back) : 0.0f;
        }
    }
}
template <class T, int N>
__device__ __forceinline__ void row_steps(float (&r)[N], const T* p, int64_t t, int64_t end) {
    if (t + N <= end) {
        const VecN<T, N> v = *reinterpret_cast<const VecN<T, N>*>(p + t);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = to_f(v.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = t + i < end ? to_f(p[t + i]) : 0.0f;
    }
}
template <class T>
__device__ __forceinline__ void put_row(const float (&r)[8], T* p, int64_t t, int64_t end) {
    if (t + 8 <= end) {
        Vec8<T> v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v.v[i] = from_f<T>(r[i]);
        *reinterpret_cast<Vec8<T>*>(p + t) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + i < end) p[t + i] = from_f<T>(r[i]);
    }
}

template <class T, int W>
__global__ __launch_bounds__(256) void conv_rows_kernel(ConvArgs a, Geometry geo) {
    const int cb = blockIdx.x % geo.blocks;
    Item it;
    if (!find_item(a.q, blockIdx.x / geo.blocks, geo.Q, it) || it.state < 0) return;
    const int x = threadIdx.x & (geo.cx - 1);
    const int64_t h = (int64_t)cb * (256 / geo.cx) + threadIdx.x / geo.cx;
    if (h >= a.H) return;
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = a.weight[h * W + k];
    const float b = a.bias ? a.bias[h] : 0.0f;
    const T* u = (const T*)a.u.data + it.row * a.u.sb + h * a.u.sh;
    T* y = (T*)a.y.data + it.row * a.y.sb + h * a.y.sh;
    const int64_t t = (int64_t)it.beg + (int64_t)it.c * geo.Q + x * 8;
    float v[12] = {}, lo[4], hi[8];
    if (t < it.end) {
        row_before<T, W>(lo, u, t, it, (const T*)a.state_in, a.H, (int)h);
        row_steps<T, 8>(hi, u, t, it.end);
#pragma unroll
        for (int i = 0; i < 12; ++i) v[i] = i < 4 ? lo[i] : hi[i - 4];
    }
    if (it.c == 0 && x == 0) hand_on<T, W>(a, it, (int)h);
    if (t >= it.end) return;
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float acc = b;
#pragma unroll
        for (int k = 0; k < W; ++k) acc = fmaf(w[k], v[i + 4 - (W - 1) + k], acc);
        o[i] = a.silu ? silu_f<kFine<T>>(acc) : acc;
    }
    put_row<T>(o, y, t, it.end);
}

// ---- backward ----

// gradient that the final state's gradient hands to input `t` (0 <= t < len), or
// to the old input at state index j = W - 1 + t for t < 0
template <int W>
__device__ __forceinline__ float from_final(const ConvGradArgs& a, const Item& it, int64_t h, int64_t t) {
    if (!a.dstate_out) return 0.0f;
    const int64_t j = t - (it.end - it.beg) + (W - 1);
    return j >= 0 && j < W - 1 ? a.dstate_out[(it.state * a.f.H + h) * (W - 1) + j] : 0.0f;
}

// gradient of the state before the sequence: old input i (i = 0 oldest) stands
// W - 1 - i steps before step 0
template <class T, int W>
__device__ __forceinline__ void grad_old(const ConvGradArgs& a, const Item& it, int64_t h) {
    if constexpr (W > 1) {
        if (!a.dstate_in) return;
        const T* u = (const T*)a.f.u.data + it.row * a.f.u.sb + h * a.f.u.sh;
        const T* dy = (const T*)a.dy.data + it.row * a.dy.sb + h * a.dy.sh;
        const int len = it.end - it.beg;
        float line[2 * (W - 1)];  // the inputs from W - 1 steps before the sequence to W - 2 behind its first
#pragma unroll
        for (int i = 0; i < 2 * (W - 1); ++i) {
            const int t = i - (W - 1);
            line[i] = t < 0 ? old_input<T, W>((const T*)a.f.state_in, it.state, a.f.H, (int)h, -t)
                            : t < len ? to_f(u[(it.beg + t) * a.f.u.sl]) : 0.0f;
        }
        float d[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) d[i] = from_final<W>(a, it, h, i - (W - 1));
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {  // the steps whose window reaches back over the start
            float pre = a.f.bias ? a.f.bias[h] : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) pre = fmaf(a.f.weight[h * W + k], line[t + k], pre);
            const float g = t < len ? to_f(dy[(it.beg + t) * a.dy.sl]) : 0.0f;
            const float dpre = t < len ? (a.f.silu ? g * silu_slope<kFine<T>>(pre) : g) : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (t + k < W - 1) d[t + k < W - 1 ? t + k : 0] += a.f.weight[h * W + k] * dpre;
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) a.dstate_in[(it.state * a.f.H + h) * (W - 1) + i] = d[i];
    }
}

template <class T, int W, int V>
__global__ __launch_bounds__(256) void conv_grad_tokens_kernel(ConvGradArgs g, Geometry geo, float* partial) {
    __shared__ float red[256 * V];
    const ConvArgs& a = g.f;
    const int cb = blockIdx.x % geo.blocks;
    const int64_t item = blockIdx.x / geo.blocks;
    Item it;
    const bool there = find_item(a.q, item, geo.Q, it);
    const int cx = threadIdx.x & (geo.cx - 1), seg = threadIdx.x / geo.cx;
    const int64_t h = ((int64_t)cb * geo.cx + cx) * V;
    const int n = (int)max((int64_t)0, min((int64_t)V, a.H - h));
    float dw[W][V] = {}, db[V] = {};
    if (there && n > 0) {
        const int64_t first = (int64_t)it.beg + (int64_t)it.c * geo.Q + seg * geo.walk;
        const int64_t last = min((int64_t)it.end, first + geo.walk);
        const T* u = (const T*)a.u.data + it.row * a.u.sb + h * a.u.sh;
        const T* dy = (const T*)g.dy.data + it.row * g.dy.sb + h * g.dy.sh;
        T* du = (T*)g.du.data + it.row * g.du.sb + h * g.du.sh;
        if (it.c == 0 && seg == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) grad_old<T, W>(g, it, h + i);
        }
        if (first < last) {
            float w[W][V], b[V], past[W > 1 ? W - 1 : 1][V], ahead[W][V] = {};
            load_weights<W, V>(w, b, a.weight, a.bias, h, n);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                const int64_t t = first - (W - 1) + k;
                if (t >= it.beg) {
                    load_v<T, V>(past[k], u + t * a.u.sl, a.u.sh, n);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        past[k][i] = i < n ? old_input<T, W>((const T*)a.state_in, it.state, a.H, (int)h + i,
                                                             (int)(it.beg - t))
                                           : 0.0f;
                }
            }
            // ahead[j]: the gradient collected so far for input t - (W - 1) + j; the
            // walk goes W - 1 steps past `last` so that the own inputs get all theirs
            const int64_t stop = last + W - 1, there_to = min(stop, (int64_t)it.end);
            // one step: `x` and `d` the input and the gradient of y at step t (0 behind the sequence)
            auto step = [&](int64_t t, const float (&x)[V], float (&d)[V]) {
                const bool mine = t < last;
                float o[V];
                if (a.silu) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float pre = b[i];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) pre = fmaf(w[k][i], past[k][i], pre);
                        pre = fmaf(w[W - 1][i], x[i], pre);
                        d[i] *= silu_slope<kFine<T>>(pre);
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (mine) {
                        db[i] += d[i];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][i] = fmaf(d[i], past[k][i], dw[k][i]);
                        dw[W - 1][i] = fmaf(d[i], x[i], dw[W - 1][i]);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) ahead[j][i] = fmaf(w[j][i], d[i], ahead[j][i]);
                    o[i] = ahead[0][i];
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) ahead[j][i] = ahead[j + 1][i];
                    ahead[W - 1][i] = 0.0f;
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; ++k) past[k][i] = past[k + 1][i];
                    if (W > 1) past[W > 1 ? W - 2 : 0][i] = x[i];
                }
                const int64_t done = t - (W - 1);  // this input's gradient is whole
                if (done >= first) {
                    if (g.dstate_out && done >= it.end - (W - 1)) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (i < n) o[i] += from_final<W>(g, it, h + i, done - it.beg);
                    }
                    store_v<T, V>(o, du + done * g.du.sl, g.du.sh, n);
                }
            };
            int64_t t = first;
            if (V > 1 && n == V) {
                const T *fu = u + first * a.u.sl, *fd = dy + first * g.dy.sl;
                for (; t + kAhead <= there_to; t += kAhead) {
                    VecN<T, V> ru[kAhead], rd[kAhead];
#pragma unroll
                    for (int s = 0; s < kAhead; ++s, fu += a.u.sl, fd += g.dy.sl) {
                        ru[s] = *reinterpret_cast<const VecN<T, V>*>(fu);
                        rd[s] = *reinterpret_cast<const VecN<T, V>*>(fd);
                    }
#pragma unroll
                    for (int s = 0; s < kAhead; ++s) {
                        float x[V], d[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) x[i] = to_f(ru[s].v[i]), d[i] = to_f(rd[s].v[i]);
                        step(t + s, x, d);
                    }
                }
            }
            for (; t < stop; ++t) {
                float x[V] = {}, d[V] = {};
                if (t < it.end) {
                    load_v<T, V>(x, u + t * a.u.sl, a.u.sh, n);
                    load_v<T, V>(d, dy + t * g.dy.sl, g.dy.sh, n);
                    step(t, x, d);
                } else {
                    // behind the sequence nothing is added; the gradients collected come out
                    const int64_t done = t - (W - 1);
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        o[i] = ahead[0][i];
#pragma unroll
                        for (int j = 0; j + 1 < W; ++j) ahead[j][i] = ahead[j + 1][i];
                        ahead[W - 1][i] = 0.0f;
                    }
                    if (done >= first) {
                        if (g.dstate_out && done >= it.end - (W - 1)) {
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                if (i < n) o[i] += from_final<W>(g, it, h + i, done - it.beg);
                        }
                        store_v<T, V>(o, du + done * g.du.sl, g.du.sh, n);
                    }
                }
            }
        }
    }
    if (!partial) return;
    // sum over the workgroup's stretches of steps in order, then one row per workgroup
    float* out = partial + item * a.H * (W + 1);
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) red[i * 256 + threadIdx.x] = k < W ? dw[k < W ? k : 0][i] : db[i];
        __syncthreads();
        if (seg == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) {
                    float s = 0.0f;
                    for (int j = 0; j < 256 / geo.cx; ++j) s += red[i * 256 + j * geo.cx + cx];
                    out[(int64_t)k * a.H + h + i] = s;
                }
        }
    }
}

template <class T, int W>
__global__ __launch_bounds__(256) void conv_grad_rows_kernel(ConvGradArgs g, Geometry geo, float* partial) {
    __shared__ float red[(W + 1) * 256];
    const ConvArgs& a = g.f;
    const int cb = blockIdx.x % geo.blocks;
    const int64_t item = blockIdx.x / geo.blocks;
    Item it;
    const bool there = find_item(a.q, item, geo.Q, it);
    const int x = threadIdx.x & (geo.cx - 1);
    const int64_t h = (int64_t)cb * (256 / geo.cx) + threadIdx.x / geo.cx;
    float dw[W] = {}, db = 0.0f;
    if (there && h < a.H) {
        const T* u = (const T*)a.u.data + it.row * a.u.sb + h * a.u.sh;
        const T* dy = (const T*)g.dy.data + it.row * g.dy.sb + h * g.dy.sh;
        T* du = (T*)g.du.data + it.row * g.du.sb + h * g.du.sh;
        if (it.c == 0 && x == 0) grad_old<T, W>(g, it, h);
        float w[W];
#pragma unroll
        for (int k = 0; k < W; ++k) w[k] = a.weight[h * W + k];
        const float b = a.bias ? a.bias[h] : 0.0f;
        const int64_t from = (int64_t)it.beg + (int64_t)it.c * geo.Q;
        const int64_t to = min((int64_t)it.end, from + geo.Q);
        for (int64_t t = from + x * 8; t < to; t += geo.cx * 8) {
            float lo[4], mid[8], hi[4], dm[8], dh[4], v[16], d[12];
            row_before<T, W>(lo, u, t, it, (const T*)a.state_in, a.H, (int)h);
            row_steps<T, 8>(mid, u, t, it.end);
            row_steps<T, 4>(hi, u, t + 8, it.end);
            row_steps<T, 8>(dm, dy, t, it.end);
            row_steps<T, 4>(dh, dy, t + 8, it.end);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = i < 4 ? lo[i] : i < 12 ? mid[i - 4] : hi[i - 12];
#pragma unroll
            for (int i = 0; i < 12; ++i) d[i] = i < 8 ? dm[i] : dh[i - 8];  // 0 behind the sequence
#pragma unroll
            for (int i = 0; i < 8 + W - 1; ++i) {
                if (a.silu) {
                    float pre = b;
#pragma unroll
                    for (int k = 0; k < W; ++k) pre = fmaf(w[k], v[i + 4 - (W - 1) + k], pre);
                    d[i] = t + i < it.end ? d[i] * silu_slope<kFine<T>>(pre) : 0.0f;
                }
                if (i < 8) {
                    db += d[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k] = fmaf(d[i], v[i + 4 - (W - 1) + k], dw[k]);
                }
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < W; ++j) s = fmaf(w[W - 1 - j], d[i + j], s);
                o[i] = s;
            }
            if (g.dstate_out && t + 8 > it.end - (W - 1)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += from_final<W>(g, it, h, t + i - it.beg);
            }
            put_row<T>(o, du, t, it.end);
        }
    }
    if (!partial) return;
#pragma unroll
    for (int k = 0; k <= W; ++k) red[k * 256 + threadIdx.x] = k < W ? dw[k < W ? k : 0] : db;
    for (int half = geo.cx >> 1; half > 0; half >>= 1) {
        __syncthreads();
        if (x < half) {
#pragma unroll
            for (int k = 0; k <= W; ++k) red[k * 256 + threadIdx.x] += red[k * 256 + threadIdx.x + half];
        }
    }
    if (x == 0 && h < a.H) {
        float* out = partial + item * a.H * (W + 1);
#pragma unroll
        for (int k = 0; k <= W; ++k) out[(int64_t)k * a.H + h] = red[k * 256 + threadIdx.x];
    }
}

// dweight[h, k] and dbias[h] from the rows of partial sums [rows][W + 1][H]
constexpr int kSumCols = 32, kSumRows = 8;
__global__ __launch_bounds__(256) void conv_grad_sum_kernel(const float* partial, int64_t rows, int64_t H, int W,
                                                            float* dweight, float* dbias) {
    __shared__ double red[kSumRows][kSumCols];
    const int c = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    const int64_t cols = H * (W + 1), col = (int64_t)blockIdx.x * kSumCols + c;
    double s = 0.0;
    if (col < cols)
        for (int64_t i = r; i < rows; i += kSumRows) s += (double)partial[i * cols + col];
    red[r][c] = s;
    __syncthreads();
    if (r == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) s += red[i][c];
        const int64_t k = col / H, h = col % H;
        if (k < W) {
            if (dweight) dweight[h * W + k] = (float)s;
        } else if (dbias) {
            dbias[h] = (float)s;
        }
    }
}

int pow2_at_least(int64_t v, int most) {
    int p = 1;
    while (p < v && p < most) p <<= 1;
    return p;
}

template <class T>
constexpr int vec() { return 16 / (int)sizeof(T); }

// `rows`: batch rows (one when packed)
Geometry geometry(Order o, int V, int64_t H, int64_t L, int64_t rows, int iters) {
    Geometry g;
    g.walk = 0;
    if (o == kRows) {
        g.cx = pow2_at_least((L + 7) / 8, 64);
        const int64_t units = (L + g.cx * 8 - 1) / (g.cx * 8), items = (units + iters - 1) / iters;
        g.Q = g.cx * 8 * (int)((units + items - 1) / items);  // up to `iters` units, shared evenly
        const int chans = 256 / g.cx;
        g.blocks = (int)((H + chans - 1) / chans);
    } else {
        const int64_t n = (H + V - 1) / V;
        g.cx = pow2_at_least(n, 64);
        g.blocks = (int)((n + g.cx - 1) / g.cx);
        // a walk reads W - 1 steps more than it has: the longest that still gives kMany
        // workgroups, and no shorter than what is loaded together.  bf16, width 4: 4 rows
        // of 4096 channels x 2048 steps 27.0 us with kMany = 512, 28.4 with 1024, 30.4
        // with 2048; their gradients 49.6, 49.0, 54.8 (walks of up to 32: 54.9)
        constexpr int64_t kMany = 512;
        g.walk = kMaxWalk;
        while (g.walk > kAhead && rows * g.blocks * ((L + 256 / g.cx * g.walk - 1) / (256 / g.cx * g.walk)) < kMany)
            g.walk >>= 1;
        g.Q = 256 / g.cx * g.walk;
    }
    return g;
}

// batch rows for geometry()
int64_t rows_of(const Seqs& q) { return q.offsets ? 1 : q.S; }

// the backward pass by rows adds its sums up once per workgroup, over up to four units
// of steps (bf16, 4 x 2048 x 4096, width 4: 62 us, one unit 75, eight 69)
constexpr int kGradIters = 4;
constexpr int kGradV = 2;  // 96 registers, 5 waves per SIMD (4 channels: 151 and 3)

template <class T, int W>
hipError_t forward_as(const ConvArgs& a, hipStream_t s) {
    const View3* views[] = {&a.u, &a.y};
    const Order o = order_of(views, 2, 4);
    const int V = o == kTokens ? vec<T>() : 1;
    const Geometry geo = geometry(o, V, a.H, a.q.L, rows_of(a.q), 1);
    const int64_t wgs = item_count(a.q, geo.Q) * geo.blocks;
    if (!grid_fits(wgs, 256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), wg(256);
    if (o == kRows)
        conv_rows_kernel<T, W><<<grid, wg, 0, s>>>(a, geo);
    else if (o == kTokens)
        conv_tokens_kernel<T, W, vec<T>()><<<grid, wg, 0, s>>>(a, geo);
    else
        conv_tokens_kernel<T, W, 1><<<grid, wg, 0, s>>>(a, geo);
    return hipGetLastError();
}

template <class T, int W>
hipError_t backward_as(const ConvGradArgs& g, float* partial, hipStream_t s) {
    const ConvArgs& a = g.f;
    const View3* views[] = {&a.u, &g.dy, &g.du};
    const Order o = order_of(views, 3, 4);
    const int V = o == kTokens ? kGradV : 1;
    const Geometry geo = geometry(o, V, a.H, a.q.L, rows_of(a.q), kGradIters);
    const int64_t items = item_count(a.q, geo.Q), wgs = items * geo.blocks;
    if (!grid_fits(wgs, 256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), wg(256);
    float* to = g.dweight || g.dbias ? partial : nullptr;
    if (o == kRows)
        conv_grad_rows_kernel<T, W><<<grid, wg, 0, s>>>(g, geo, to);
    else if (o == kTokens)
        conv_grad_tokens_kernel<T, W, kGradV><<<grid, wg, 0, s>>>(g, geo, to);
    else
        conv_grad_tokens_kernel<T, W, 1><<<grid, wg, 0, s>>>(g, geo, to);
    if (to) {
        const int64_t cols = a.H * (W + 1);
        conv_grad_sum_kernel<<<dim3((unsigned)((cols + kSumCols - 1) / kSumCols)), wg, 0, s>>>(to, items, a.H, W,
                                                                                             g.dweight, g.dbias);
    }
    return hipGetLastError();
}

template <class T>
hipError_t forward_of(const ConvArgs& a, hipStream_t s) {
    switch (a.width) {
        case 1: return forward_as<T, 1>(a, s);
        case 2: return forward_as<T, 2>(a, s);
        case 3: return forward_as<T, 3>(a, s);
        default: return forward_as<T, 4>(a, s);
    }
}
template <class T>
hipError_t backward_of(const ConvGradArgs& g, float* partial, hipStream_t s) {
    switch (g.f.width) {
        case 1: return backward_as<T, 1>(g, partial, s);
        case 2: return backward_as<T, 2>(g, partial, s);
        case 3: return backward_as<T, 3>(g, partial, s);
        default: return backward_as<T, 4>(g, partial, s);
    }
}

}  // namespace

// partial sums of the weights' gradients; the largest over the storage orders
size_t conv_grad_workspace_bytes(const Seqs& q, int64_t H, int width) {
    int64_t items = 0;
    for (Order o : {kRows, kTokens, kAny})
        for (int V : {1, kGradV}) {
            const int64_t n = item_count(q, geometry(o, V, H, q.L, rows_of(q), kGradIters).Q);
            items = n > items ? n : items;
        }
    return (size_t)items * H * (width + 1) * sizeof(float);
}

// whether every storage order's launch can be made
bool conv_fits(const Seqs& q, int64_t H) {
    for (Order o : {kRows, kTokens, kAny})
        for (int V : {1, kGradV, 4, 8}) {
            const Geometry g = geometry(o, V, H, q.L, rows_of(q), 1);
            if (!grid_fits(item_count(q, g.Q) * g.blocks, 256)) return false;
        }
    return grid_fits((H * (4 + 1) + kSumCols - 1) / kSumCols, 256);
}

hipError_t launch_causal_conv(int dtype, const ConvArgs& a, hipStream_t s) {
    if (dtype == SSM_F32) return forward_of<float>(a, s);
    if (dtype == SSM_BF16) return forward_of<bf16>(a, s);
    return forward_of<f16>(a, s);
}

hipError_t launch_causal_conv_backward(int dtype, const ConvGradArgs& g, void* ws, hipStream_t s) {
    if (dtype == SSM_F32) return backward_of<float>(g, (float*)ws, s);
    if (dtype == SSM_BF16) return backward_of<bf16>(g, (float*)ws, s);
    return backward_of<f16>(g, (float*)ws, s);
}

}  // namespace ssm

// Shared pieces of the linear attention kernels: fragments of the matrix
// instructions, tiles of a chunk in LDS, and the argument blocks.
#pragma once

#include <type_traits>

#include "selective.hpp"

namespace ssm {

using f32x4 = float __attribute__((ext_vector_type(4)));
using i16x4 = short __attribute__((ext_vector_type(4)));
using i16x8 = short __attribute__((ext_vector_type(8)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));
using u16x2 = unsigned short __attribute__((ext_vector_type(2)));

constexpr int64_t kMaxKeys = 256;
constexpr int64_t kMaxValues = 256;

// ---- fragments ----
// The matrix instructions take 16 rows (or columns) by 32 numbers of the summed
// axis: lane l has row l & 15 and, of the 32, the eight that belong to l >> 4 (any
// eight, the same ones in both operands).  In float32 the eight go through eight
// instructions of four numbers each.  Results: lane l has column l & 15 (of the
// second operand) and rows 4 (l >> 4) .. + 3 (of the first).
template <class T>
struct Frag {  // bf16, f16
    i16x8 v;
};
template <>
struct Frag<float> {
    float v[8];
};

template <class T>
__device__ __forceinline__ f32x4 mma(const Frag<T>& a, const Frag<T>& b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma<bf16>(const Frag<bf16>& a, const Frag<bf16>& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c,
                                                   0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<f16>(const Frag<f16>& a, const Frag<f16>& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.v), __builtin_bit_cast(f16x8, b.v), c, 0,
                                                  0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<float>(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}

template <class T>
__device__ __forceinline__ Frag<T> frag_of(const float (&x)[8]) {
    Frag<T> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = __builtin_bit_cast(short, from_f<T>(x[j]));
    return f;
}
template <>
__device__ __forceinline__ Frag<float> frag_of<float>(const float (&x)[8]) {
    Frag<float> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = x[j];
    return f;
}
template <class T>
__device__ __forceinline__ float frag_get(const Frag<T>& f, int j) {
    return to_f(__builtin_bit_cast(T, (short)f.v[j]));
}
template <>
__device__ __forceinline__ float frag_get<float>(const Frag<float>& f, int j) {
    return f.v[j];
}
// x = hi + lo to 16 (bf16) or 22 bits (f16); in float32 hi is x itself
template <class T>
__device__ __forceinline__ void split(const float (&x)[8], Frag<T>& hi, Frag<T>& lo) {
    float y[8], r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // one number for both parts: a product would be rounded to f16 in one step for the
        // first and by way of float32 for the second
        y[j] = x[j];
        asm("" : "+v"(y[j]));
    }
    hi = frag_of<T>(y);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = y[j] - frag_get<T>(hi, j);
    lo = frag_of<T>(r);
}
template <>
__device__ __forceinline__ void split<float>(const float (&x)[8], Frag<float>& hi, Frag<float>&) {
    hi = frag_of<float>(x);
}
template <class T>
constexpr bool kSplit = sizeof(T) == 2;

// ---- tiles of a chunk in LDS: one row per step, 16 bytes of room behind each ----
template <class T>
constexpr int kChunk = sizeof(T) == 2 ? 64 : 32;  // steps: tiles of the same bytes in every type
template <class T>
constexpr int kRoom = 16 / (int)sizeof(T);

// eight numbers of a row: the summed axis along the row
template <class T>
__device__ __forceinline__ Frag<T> row_frag(const T* p) {
    return {*reinterpret_cast<const i16x8*>(p)};
}
template <>
__device__ __forceinline__ Frag<float> row_frag<float>(const float* p) {
    Frag<float> f;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
    return f;
}
// four numbers at p and four at p + 16: the order in which results of two
// neighbouring tiles become an operand without an exchange between lanes
template <class T>
__device__ __forceinline__ Frag<T> pair_frag(const T* p) {
    const i16x4 a = *reinterpret_cast<const i16x4*>(p), b = *reinterpret_cast<const i16x4*>(p + 16);
    return {__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7)};
}
template <>
__device__ __forceinline__ Frag<float> pair_frag<float>(const float* p) {
    Frag<float> f;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
    return f;
}
// eight steps of a column: the summed axis down the rows.  Sixteen lanes read four
// rows of sixteen numbers and get a column each (ds_read_b64_tr_b16); every lane of
// the wave takes part.  `p`: the tile's column 0 of the 16, row 0 of the 32.
template <class T>
__device__ __forceinline__ Frag<T> column_frag(const T* p, int stride, int lane) {
    using Half = __attribute__((address_space(3))) i16x4;
    const int g = lane >> 4, i = lane & 15;
    const T* at = p + (8 * g + (i >> 2)) * stride + 4 * (i & 3);
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Half*)at);
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Half*)(at + 4 * stride));
    return {__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7)};
}
template <>
__device__ __forceinline__ Frag<float> column_frag<float>(const float* p, int stride, int lane) {
    Frag<float> f;
    const float* at = p + 8 * (lane >> 4) * stride + (lane & 15);
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = at[j * stride];
    return f;
}

// how a tensor [steps, columns] lies
enum Lay : int { kByColumn, kByStep, kElement };  // columns contiguous, steps contiguous, neither
inline Lay lay_of(const View4& v) { return v.sn == 1 ? kByColumn : v.sl == 1 ? kByStep : kElement; }

// A chunk's tile on its way from memory to LDS: columns CP (those behind the last one and
// steps behind the chunk's `nt` are zero), TH threads, each with vectors of 16 bytes along
// whichever axis is contiguous.
template <class T, int CP, int TH>
struct Carrier {
    static constexpr int Q = kChunk<T>, V = kRoom<T>, K = Q * CP / (TH * V), kStride = CP + kRoom<T>;
    static_assert(Q * CP % (TH * V) == 0, "whole vectors");
    using Vec = typename std::conditional<sizeof(T) == 2, Vec8<T>, Vec4<T>>::type;
    Vec r[K];

    static __device__ __forceinline__ void place(Lay lay, int tid, int k, int& step, int& col) {
        const int e = tid + TH * k;
        if (lay == kByStep) {
            step = e % (Q / V) * V;
            col = e / (Q / V);
        } else {
            step = e / (CP / V);
            col = e % (CP / V) * V;
        }
    }
    // `p`: the chunk's first step, column 0; C columns exist
    __device__ __forceinline__ void load(const T* p, Lay lay, int64_t sn, int64_t sl, int C, int nt, int tid) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int step, col;
            place(lay, tid, k, step, col);
            const T* at = p + step * sl + col * sn;
            const bool by_step = lay == kByStep;
            const int there = by_step ? (col < C ? nt - step : 0) : (step < nt ? C - col : 0);
            if (there >= V && lay != kElement) {
                r[k] = *reinterpret_cast<const Vec*>(at);
            } else {
                const int64_t d = by_step ? 1 : sn;
#pragma unroll
                for (int i = 0; i < V; ++i) r[k].v[i] = i < there ? at[i * d] : from_f<T>(0.0f);
            }
        }
    }
    // row of step i: i, or from the chunk's end
    template <bool REVERSE>
    __device__ __forceinline__ void store(T* to, Lay lay, int tid) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int step, col;
            place(lay, tid, k, step, col);
            if (lay == kByStep) {
#pragma unroll
                for (int i = 0; i < V; ++i) to[(REVERSE ? Q - 1 - step - i : step + i) * kStride + col] = r[k].v[i];
            } else {
                *reinterpret_cast<f32x4*>(to + (REVERSE ? Q - 1 - step : step) * kStride + col) =
                    __builtin_bit_cast(f32x4, r[k]);
            }
        }
    }
    // the largest magnitude as bits: at or above kInf<T> where one is infinite or NaN
    __device__ __forceinline__ uint32_t most() const {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 2) {
            u16x2 w = {0, 0};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                struct Words { uint32_t w[4]; };
                const Words x = __builtin_bit_cast(Words, r[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w = __builtin_elementwise_max(w, __builtin_bit_cast(u16x2, x.w[i] & 0x7fff7fffu));
            }
            m = max((uint32_t)w[0], (uint32_t)w[1]);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(to_f(r[k].v[i])) & 0x7fffffffu);
        }
        return m;
    }
};
template <class T>
constexpr uint32_t kInf = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, f16>::value ? 0x7c00u : 0x7f80u;

// A power of two 2^e that brings magnitudes up to `most` (float32) below 2^15, where
// float16 has them and 2^-39 of them; 1 for other types.  Bounded, so that it and its
// reciprocal are float32.
template <class T>
__device__ __forceinline__ float to_range(float most) {
    if constexpr (!std::is_same<T, f16>::value) return 1.0f;
    const int e = 127 + 14 - (int)((__float_as_uint(most) >> 23) & 0xff);  // 14 - floor(log2 most)
    return most > 0.0f ? __uint_as_float((uint32_t)(min(max(e, -110), 110) + 127) << 23) : 1.0f;
}
// 1 / a power of two
__device__ __forceinline__ float reciprocal_of_power(float p) {
    return __uint_as_float((254u << 23) - __float_as_uint(p));
}

template <int CTRL>
__device__ __forceinline__ float dpp_zero(float v) {  // lanes without a source get 0
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// sums over the 16 lanes of a row, in every lane
__device__ __forceinline__ float row_sum(float v) {
    v += dpp<0xB1>(v);    // lanes 1 apart
    v += dpp<0x4E>(v);    // 2
    v += dpp<0x141>(v);   // the other quad of eight
    return v + dpp<0x140>(v);
}
// sums over lanes 16 and 32 apart, in every lane
__device__ __forceinline__ float across_rows(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// ---- decays of a chunk ----
// With g_r the log decay of row r, the weight of the pair (t, s), s <= t, is
// exp(g_{s+1} + .. + g_t).  It is never the quotient of two running products: those
// lose the value where one of them is small, and an infinite g (a reset) would give
// infinity less infinity.  Rows are taken in blocks of 16: across blocks the weight is
// exp(sum to the end of s's block) exp(sum of the blocks between) exp(sum within t's),
// each a sum of terms that are there; within a block the sums are formed pair by pair.
template <class T>
struct Decays {
    static constexpr int Q = kChunk<T>, B = Q / 16;
    float g[Q], in[Q], out[Q];     // of each row: log decay, weight towards the state, weight of what is read
    float head[Q], tail[Q];        // exp(sum from t's block's start to t) out_t; exp(sum behind s to its block's end) in_s
    float from[Q], to[Q];          // the same from the chunk's start, to its end
    float between[B][B];           // [i][j]: exp(sum over the blocks between j < i)
    float whole;                   // exp(sum of all)
    float most_in, most_out, grow; // largest weights; at least as much as any product of decays (float16 only)
    int odd;                       // the chunk has to be walked step by step
};
// one wave, lane r (of Q) with row r's values
template <class T>
__device__ __forceinline__ void put_decays(Decays<T>& d, float g, float in, float out, int lane) {
    constexpr int Q = kChunk<T>, B = Q / 16;
    const bool row = lane < Q;
    g = row ? g : 0.0f, in = row ? in : 0.0f, out = row ? out : 0.0f;
    float pre = g, suf = dpp_zero<0x101>(g);
    pre += dpp_zero<0x111>(pre), suf += dpp_zero<0x101>(suf);
    pre += dpp_zero<0x112>(pre), suf += dpp_zero<0x102>(suf);
    pre += dpp_zero<0x114>(pre), suf += dpp_zero<0x104>(suf);
    pre += dpp_zero<0x118>(pre), suf += dpp_zero<0x108>(suf);
    float sum[B], before = 0.0f, after = 0.0f, all = 0.0f;
    const int block = lane >> 4;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        sum[b] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(pre), 16 * b + 15));
        before += b < block ? sum[b] : 0.0f;
        after += b > block ? sum[b] : 0.0f;
        all += sum[b];
    }
    constexpr bool F = kFine<T>;
    if (row) {
        d.g[lane] = g, d.in[lane] = in, d.out[lane] = out;
        d.head[lane] = exp_f<F>(pre) * out;
        d.tail[lane] = exp_f<F>(suf) * in;
        d.from[lane] = exp_f<F>(before + pre) * out;
        d.to[lane] = exp_f<F>(suf + after) * in;
    }
    if (lane < B * B) {
        const int i = lane / B, j = lane % B;
        float m = 0.0f;
#pragma unroll
        for (int b = 0; b < B; ++b) m += b > j && b < i ? sum[b] : 0.0f;
        d.between[i][j] = exp_f<F>(m);
    }
    // growth that could pass the type's range in a part of a product, NaN or infinite weights
    constexpr bool H = std::is_same<T, f16>::value;
    const float up = across_rows(row_sum(fmaxf(g, 0.0f)));
    const bool odd = !(up < (H ? 4.0f : 40.0f)) || __ballot(g != g || !(fabsf(in) < INFINITY) || !(fabsf(out) < INFINITY));
    if (lane == 0) {
        d.whole = exp_f<F>(all);
        d.odd = odd;
        if (H) d.grow = exp_f<F>(up);
    }
    if constexpr (H) {
        float a = fabsf(in), b = fabsf(out);
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) a = fmaxf(a, __shfl_xor(a, k)), b = fmaxf(b, __shfl_xor(b, k));
        if (lane == 0) d.most_in = a, d.most_out = b;
    }
}
// the weights out_t E in_s of lane's elements of tile (ti, si): t = 16 ti + (lane & 15),
// s = 16 si + 4 (lane >> 4) + i; zero for s > t
template <class T>
__device__ __forceinline__ f32x4 pair_weights(const Decays<T>& d, int ti, int si, int lane) {
    const int tl = lane & 15, gl = lane >> 4, t = 16 * ti + tl, s = 16 * si + 4 * gl;
    f32x4 r;
    if (ti != si) {
        const float b = d.between[ti][si];
        const f32x4 v = *reinterpret_cast<const f32x4*>(&d.tail[s]);
        const float h = d.head[t] * b;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = h * v[i];
        return r;
    }
    f32x4 q[4];
    float sums[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        q[b] = *reinterpret_cast<const f32x4*>(&d.g[16 * ti + 4 * b]);
        sums[b] = (q[b][0] + q[b][1]) + (q[b][2] + q[b][3]);
    }
    const int tb = tl >> 2, tr = tl & 3;
    const bool same = tb == gl;
    // t's own four up to t, s's four behind s (up to t where both are the same), those between
    const f32x4 qt = tb == 0 ? q[0] : tb == 1 ? q[1] : tb == 2 ? q[2] : q[3];
    f32x4 qs = gl == 0 ? q[0] : gl == 1 ? q[1] : gl == 2 ? q[2] : q[3];
    float rest = qt[0] + (tr > 0 ? qt[1] : 0.0f) + (tr > 1 ? qt[2] : 0.0f) + (tr > 2 ? qt[3] : 0.0f);
    rest += (gl < 1 && tb > 1 ? sums[1] : 0.0f) + (gl < 2 && tb > 2 ? sums[2] : 0.0f);
    rest = same ? 0.0f : rest;
#pragma unroll
    for (int i = 1; i < 4; ++i) qs[i] = same && i > tr ? 0.0f : qs[i];
    float e[4];
    e[3] = rest;
    e[2] = rest + qs[3];
    e[1] = rest + (qs[2] + qs[3]);
    e[0] = rest + (qs[1] + (qs[2] + qs[3]));
    const float o = d.out[t];
    const f32x4 w = *reinterpret_cast<const f32x4*>(&d.in[s]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = s + i <= t ? exp_f<kFine<T>>(e[i]) * (o * w[i]) : 0.0f;
    return r;
}

// ---- argument blocks ----
// One walk over the chunks of every sequence: with x the state before a row,
//   x <- exp(g) x + in key value^T,  result = out (x^T query) + D value.
// Forwards: key k, query q, value v, in beta, out scale.  Backwards (REVERSE), with g
// of the step behind: key q, query k, value dy, in scale, out beta; the result is dv.
struct WalkArgs {
    Seqs q;
    int64_t H, G, N, P;
    View4 key, query, value, result;  // result.data null: the states alone
    Lay key_lay, query_lay, value_lay;
    View3 g, beta;                    // float; beta.data nullable
    float scale;
    const float* D;                   // [H] nullable
    const float* x_in;                // [states, H, N, P] nullable
    float* x_out;                     // nullable
    float* saved;                     // nullable: the states before every chunk
    int64_t segment;                  // steps of a segment, whole chunks
    int64_t items;                    // segments of all sequences
    float* seg_x;                     // [items, H, N, P]: what a segment leaves of a state of zero (the first: of x_in)
    float* seg_decay;                 // [items, H]
};

struct LinearArgs {
    Seqs q;
    int64_t Bsz, H, G, N, P;
    float scale;
    View4 qv, k, v, y;  // qv: the queries
    View3 g, beta;
    const float *D, *x_in;
    float *x_out, *saved;
};

struct LinearGradArgs {
    LinearArgs f;  // the forward call's (y, x_out unused)
    View4 dy, dq, dk, dv;
    View3 dg, dbeta;         // float; dbeta nullable
    float *dD, *dx_in;       // nullable
    const float* dx_out;     // nullable
};

// what the pairs' kernel takes: the forward call's tensors, the states before every chunk
// and the gradients of the states behind them, both [rows, H, N, padded P]
struct PairArgs {
    Seqs q;
    int64_t Bsz, H, G, N, P;
    float scale;
    View4 qv, k, v, dy, dq, dk;
    Lay q_lay, k_lay, v_lay, dy_lay;
    View3 g, beta, dg, dbeta;  // beta, dbeta nullable
    const float *states, *ahead;
    int heads, blocks;         // heads of a workgroup, workgroups of a group
    int64_t items;             // chunks of all sequences
    float* parts;              // blocks > 1: [blocks, 2, Bsz, G, L, N], sums over a block's heads
    float* skips;              // [items, H]: dy . v over a chunk; null without D
    float* dD;
};

struct LinearStepArgs {
    int64_t Bsz, H, G, N, P;
    float scale;
    const int32_t* slots;
    int64_t n_slots;
    const void *q, *k, *v;
    void* y;
    int64_t q_row, q_group, q_key, k_row, k_group, k_key, v_row, v_head, v_value, y_row, y_head, y_value;
    const float *g, *beta;  // beta nullable
    int64_t g_row, g_head, beta_row, beta_head;
    const float* D;
    float* x;
};

// The states kept for the backward pass, one before every chunk: row (first of the
// sequence + chunk) of [rows, H, N, padded P]
inline int64_t padded_values(int64_t P) { return (P + 31) / 32 * 32; }
__host__ __device__ inline int64_t linear_rows(int64_t S, int64_t L, bool packed, int Q) {
    return packed ? L / Q + S : S * ((L + Q - 1) / Q);
}
__device__ __forceinline__ int64_t linear_row(const Seqs& q, const Item& it, int Q) {
    return q.offsets ? (int64_t)(it.beg / Q) + it.s : (int64_t)it.s * ((q.L + Q - 1) / Q);
}

}  // namespace ssm

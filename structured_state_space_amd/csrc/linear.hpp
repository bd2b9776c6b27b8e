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
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
// 16 bytes anywhere that the element's alignment allows
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Words {
    u32x4 v;
};

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

// two numbers rounded to the type, in a word
template <class T>
__device__ __forceinline__ uint32_t pack_two(float a, float b) {
    if constexpr (std::is_same<T, bf16>::value) {  // (one instruction; number by number it took one each and a third)
        using f32x2 = float __attribute__((ext_vector_type(2)));
        using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    } else {
        return __builtin_bit_cast(uint16_t, from_f<T>(a)) | (uint32_t)__builtin_bit_cast(uint16_t, from_f<T>(b)) << 16;
    }
}
template <class T>
__device__ __forceinline__ Frag<T> frag_of(const float (&x)[8]) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_two<T>(x[2 * j], x[2 * j + 1]);
    return {__builtin_bit_cast(i16x8, w)};
}
// four numbers, rounded to the type
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Quad {
    uint32_t w[sizeof(T)];
};
template <class T>
__device__ __forceinline__ Quad<T> four_of(const f32x4& x) {
    if constexpr (sizeof(T) == 4)
        return {{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])}};
    else return {{pack_two<T>(x[0], x[1]), pack_two<T>(x[2], x[3])}};
}
template <class T>
__device__ __forceinline__ T get_of(const Quad<T>& f, int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(f.w[i]);
    else return __builtin_bit_cast(T, (uint16_t)(f.w[i / 2] >> (16 * (i & 1))));
}
// in LDS, where they are aligned
template <class T>
__device__ __forceinline__ void put_four(T* at, const f32x4& x) {
    struct __attribute__((aligned(4 * sizeof(T)))) Aligned { Quad<T> v; };
    *reinterpret_cast<Aligned*>(at) = {four_of<T>(x)};
}
// The same in parts, `apart` elements from one to the next.  float16's second part is taken kLift
// times: below 2^-14 it would have ever fewer bits, and so would what is small beside the chunk's
// largest weight (2^-50 of it is kept, instead of 2^-39).
template <class T>
constexpr float kLift = std::is_same<T, f16>::value ? 0x1p11f : 1.0f;
template <class T, int K>
__device__ __forceinline__ void put_parts(T* at, int apart, f32x4 x) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        put_four<T>(at + k * apart, x);
        if (k + 1 < K) {
            const Quad<T> f = four_of<T>(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (x[i] - to_f(get_of<T>(f, i))) * kLift<T>;
        }
    }
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
// Float32 numbers as sums of operands of the type: one in float32, two in f16 (22 bits), three
// in bf16 (24 bits; two, 16 bits, left errors of 2.4e-6 in the states).
template <class T>
constexpr int kParts = sizeof(T) == 4 ? 1 : std::is_same<T, f16>::value ? 2 : 3;
// Those of the operands that only give results of the type (the weights of pairs, the state in y and
// dv): two in bf16 as well, 2^-17 of each.  In one part the results had the error of two roundings
// instead of one.
template <class T>
constexpr int kShort = sizeof(T) == 4 ? 1 : 2;
template <class T, int K>
__device__ __forceinline__ void split(const float (&x)[8], Frag<T> (&part)[K]) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // one number for both parts: a product would be rounded to f16 in one step for the
        // first and by way of float32 for the second
        r[j] = x[j];
        if (std::is_same<T, f16>::value) asm("" : "+v"(r[j]));
    }
    part[0] = frag_of<T>(r);
#pragma unroll
    for (int i = 1; i < K; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] -= frag_get<T>(part[i - 1], j);
        part[i] = frag_of<T>(r);
    }
}

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
// the first four of these, and four zeros
template <class T>
__device__ __forceinline__ Frag<T> half_frag(const T* p) {
    return {__builtin_shufflevector(*reinterpret_cast<const i16x4*>(p), i16x4{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7)};
}
template <>
__device__ __forceinline__ Frag<float> half_frag<float>(const float* p) {
    Frag<float> f;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = 0.0f;
    return f;
}
// The weights of a chunk's pairs in LDS, a row per later step: 32 rows have 32 columns, the next 32
// 64 (products take 32 at a time), with 16 bytes of room behind each.
template <class T>
struct PairPlaces {
    static constexpr int kSize = kChunk<T> / 32 == 1 ? 32 * (32 + kRoom<T>) : 32 * (96 + 2 * kRoom<T>);
    static __device__ __forceinline__ constexpr int stride(int block) { return 32 * (block + 1) + kRoom<T>; }
    // row r, which is in block r / 32
    static __device__ __forceinline__ constexpr int row(int block, int r) {
        return (block ? 32 * (32 + kRoom<T>) : 0) + (r - 32 * block) * stride(block);
    }
};
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

// How a tensor [steps, columns] is read: vectors of 16 bytes of neighbouring columns (a whole
// number of them), vectors of neighbouring steps (in whole chunks), or element by element.
enum Lay : int { kByColumn, kByStep, kElement };
// a tile of a call's tensors: strides in bytes where vectors are read
struct Source {
    const char* data = nullptr;
    int64_t sb = 0, sg = 0, sn = 0, sl = 0;  // bytes
    Lay lay = kElement;
};
inline Source source_of(const View4& v, int64_t columns, int64_t size) {
    Source s;
    s.data = (const char*)v.data;
    s.sb = v.sb * size, s.sg = v.sg * size, s.sn = v.sn * size, s.sl = v.sl * size;
    // distances within a chunk are 32 bits wide
    if (v.sn == 1 && columns % (16 / size) == 0) s.lay = kByColumn;
    else if (v.sl == 1 && s.sn < ((int64_t)1 << 24)) s.lay = kByStep;
    return s;
}

// A chunk's tile on its way from memory to LDS: columns CP (those behind the last one and
// steps behind the chunk's `nt` become zero), TH threads, each with vectors of 16 bytes.
// The loads are unconditional, at clamped places, and what does not exist is cleared when
// the tile is stored, a chunk later: conditions around the loads, vector by vector, took
// thousands of scalar instructions, and clearing at once would wait for the data.
// FAST: vectors of columns, known when the kernel is compiled.
template <class T, int CP, int TH, bool FAST>
struct Carrier {
    static constexpr int Q = kChunk<T>, V = kRoom<T>, kVectors = Q * CP / V, kStride = CP + kRoom<T>;
    static constexpr int K = kVectors > TH ? kVectors / TH : 1;
    static_assert(kVectors % TH == 0 || kVectors < TH, "a vector each, or some threads none");
    u32x4 r[K] = {};  // (whole words: element by element they took a register each)

    static __device__ __forceinline__ bool idle(int tid) { return kVectors < TH && tid >= kVectors; }

    static __device__ __forceinline__ void place(Lay lay, int tid, int k, int& step, int& col) {
        const uint32_t e = (uint32_t)tid + TH * k;
        if (lay == kByStep) {
            step = e % (Q / V) * V;
            col = e / (Q / V);
        } else {
            step = e / (CP / V);
            col = e % (CP / V) * V;
        }
    }
    // `p`: the chunk's first step, column 0; C columns and nt >= 1 steps exist
    __device__ __forceinline__ void load(const char* p, const Source& s, int C, int nt, int tid) {
        constexpr uint32_t E = sizeof(T);
        if (idle(tid)) return;
        if (FAST || s.lay == kByColumn) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                int step, col;
                place(kByColumn, tid, k, step, col);
                r[k] = reinterpret_cast<const Words<T>*>(p + ((uint32_t)min(step, nt - 1) * (uint32_t)s.sl + (uint32_t)min(col, C - V) * E))->v;
            }
        } else if (s.lay == kByStep && nt == Q) {
            const int t = anew(tid);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                int step, col;
                place(kByStep, t, k, step, col);
                r[k] = reinterpret_cast<const Words<T>*>(p + ((uint32_t)step * E + (uint32_t)min(col, C - 1) * (uint32_t)s.sn))->v;
            }
        } else {
            const int t = anew(tid);  // the addresses are worked out here, and not kept from chunk to chunk
#pragma unroll
            for (int k = 0; k < K; ++k) {
                int step, col;
                place(s.lay, t, k, step, col);
                const bool by_step = s.lay == kByStep;
                const char* at[V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    at[i] = p + min(step + (by_step ? i : 0), nt - 1) * s.sl + min(col + (by_step ? 0 : i), C - 1) * s.sn;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(T) == 4) r[k][i] = *reinterpret_cast<const uint32_t*>(at[i]);
                    else
                        r[k][i] = *reinterpret_cast<const uint16_t*>(at[2 * i]) |
                                  (uint32_t)*reinterpret_cast<const uint16_t*>(at[2 * i + 1]) << 16;
                }
            }
        }
    }
    // what does not exist becomes zero
    __device__ __forceinline__ void clear(Lay lay, int C, int nt, int tid) {
        if (FAST) lay = kByColumn;
        if (__builtin_expect(nt == Q && C >= CP, 1)) return;
        const int t = anew(tid);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int step, col;
            place(lay, t, k, step, col);
            if (lay == kByColumn) {
                const uint32_t m = step < nt && col < C ? ~0u : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) r[k][i] &= m;
            } else {
                const int there = lay == kByStep ? (col < C ? nt - step : 0) : (step < nt ? C - col : 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(T) == 4) r[k][i] &= i < there ? ~0u : 0u;
                    else r[k][i] &= 2 * i + 1 < there ? ~0u : 2 * i < there ? 0xffffu : 0u;
                }
            }
        }
    }
    // row of step i: i, or from the chunk's end
    template <bool REVERSE>
    __device__ __forceinline__ void store(T* to, Lay lay, int tid) const {
        if (FAST) lay = kByColumn;
        const int t = anew(tid);
        if (idle(t)) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int step, col;
            place(lay, t, k, step, col);
            if (lay == kByStep) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    T* at = to + (REVERSE ? Q - 1 - step - i : step + i) * kStride + col;
                    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(at) = r[k][i];
                    else *reinterpret_cast<uint16_t*>(at) = (uint16_t)(r[k][i / 2] >> (16 * (i & 1)));
                }
            } else {
                *reinterpret_cast<u32x4*>(to + __umul24(REVERSE ? Q - 1 - step : step, kStride) + col) = r[k];
            }
        }
    }
    // the largest magnitude as bits (an infinity's or NaN's are above every number's)
    __device__ __forceinline__ uint32_t most() const {
        if constexpr (sizeof(T) == 2) {
            u16x2 w = {0, 0};
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) w = __builtin_elementwise_max(w, __builtin_bit_cast(u16x2, r[k][i] & 0x7fff7fffu));
            return max((uint32_t)w[0], (uint32_t)w[1]);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = max(m, r[k][i] & 0x7fffffffu);
            return m;
        }
    }
};
// Bits of the magnitudes from which on a chunk goes row by row: 2^22 for queries and keys, 2^39 for
// values, infinity in float16.  Below, with put_decays' bounds, no product of a chunk's inputs passes
// float32: a weight of a pair stays below N 2^44 2^60 2^14 <= 2^126 and what a chunk adds to the
// state below 64 2^22 2^39 2^60 = 2^127.
template <class T>
constexpr uint32_t kHuge = sizeof(T) == 4 ? 0x4a800000u : std::is_same<T, f16>::value ? 0x7c00u : 0x4a80u;
template <class T>
constexpr uint32_t kHugeValue = sizeof(T) == 4 ? 0x53000000u : std::is_same<T, f16>::value ? 0x7c00u : 0x5300u;

// A power of two 2^e that brings magnitudes up to `most` (float32) below 2^15, where
// float16 has them and 2^-39 of them; 1 for other types.  Bounded by what float32's largest
// number needs and so that its reciprocal is float32.
template <class T>
__device__ __forceinline__ float to_range(float most) {
    if constexpr (!std::is_same<T, f16>::value) return 1.0f;
    const int e = 127 + 14 - (int)((__float_as_uint(most) >> 23) & 0xff);  // 14 - floor(log2 most)
    return most > 0.0f ? __uint_as_float((uint32_t)(min(max(e, -113), 110) + 127) << 23) : 1.0f;
}
// 1 / a power of two
__device__ __forceinline__ float reciprocal_of_power(float p) {
    return __uint_as_float((254u << 23) - __float_as_uint(p));
}

// Some of the products are infinite, NaN or beyond 2^64 (whose squares pass float32).
template <int K>
__device__ __forceinline__ bool far_out(const f32x4 (&x)[K]) {
    float all = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) all = fmaf(x[k][i], x[k][i], all);
    return !(all < INFINITY);
}

// The products of two tiles' rows where those pass float32 (lane: row l & 15 of either at its part of
// the summed axis).  Rows with a number of 2^30 or more are taken 2^-98 times: bits 0 to 15 of `rows`
// name those of `a`, bits 16 to 31 those of `b`.
constexpr float kFar = 0x1p98f;
template <class T, int KK>
__device__ __forceinline__ f32x4 products_in_range(const T* a, const T* b, uint32_t& rows) {
    auto most = [](const T* p) {
        float m = 0.0f;
        for (int kk = 0; kk < KK; ++kk) {
            const Frag<T> f = row_frag<T>(p + 32 * kk);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(frag_get<T>(f, j)));
        }
        m = fmaxf(m, __shfl_xor(m, 16));
        return fmaxf(m, __shfl_xor(m, 32));
    };
    auto taken = [](const T* p, float factor) {
        const Frag<T> f = row_frag<T>(p);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = frag_get<T>(f, j) * factor;
        return frag_of<T>(x);
    };
    const bool far_a = most(a) >= 0x1p30f, far_b = most(b) >= 0x1p30f;
    const float fa = far_a ? 1.0f / kFar : 1.0f, fb = far_b ? 1.0f / kFar : 1.0f;
    rows = (uint32_t)(__ballot(far_a) & 0xffff) | (uint32_t)(__ballot(far_b) & 0xffff) << 16;
    f32x4 c = {0, 0, 0, 0};
    for (int kk = 0; kk < KK; ++kk) c = mma<T>(taken(a + 32 * kk, fa), taken(b + 32 * kk, fb), c);
    return c;
}
// Such a product's x y of row i of `a` and row j of `b`, brought back in the smaller of the factors:
// nothing passes float32, at either end, that the whole product does not.
__device__ __forceinline__ void bring_back(float& x, float& y, uint32_t rows, int i, int j) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float f = rows >> (k ? 16 + j : i) & 1 ? kFar : 1.0f;
        const bool first = fabsf(x) < fabsf(y);
        x *= first ? f : 1.0f, y *= first ? 1.0f : f;
    }
}
// the type's largest number
template <class T>
constexpr float kLargest = std::is_same<T, f16>::value ? 65504.0f : sizeof(T) == 2 ? 0x1.fep127f : 0x1.fffffep127f;

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
// the sum over a row's lanes from this one on, and up to this one
__device__ __forceinline__ float row_suffix(float v) {
    v += dpp_zero<0x101>(v);
    v += dpp_zero<0x102>(v);
    v += dpp_zero<0x104>(v);
    return v + dpp_zero<0x108>(v);
}
__device__ __forceinline__ float row_prefix(float v) {
    v += dpp_zero<0x111>(v);
    v += dpp_zero<0x112>(v);
    v += dpp_zero<0x114>(v);
    return v + dpp_zero<0x118>(v);
}
// lane i's value, in every lane
__device__ __forceinline__ float of_lane(float v, int i) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}
// sums over lanes 16 and 32 apart, in every lane (exchanges of registers, not by way of LDS)
__device__ __forceinline__ float across_rows(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Neighbouring workgroups go to the eight dies in turn, each with a cache of its own.  The
// place of workgroup `bid` of n in an order in which a die's workgroups are neighbours.
__device__ __forceinline__ int64_t by_die(int64_t bid, int64_t n) {
    const int64_t die = bid & 7, each = n >> 3, rest = n & 7;
    return die * each + min(die, rest) + (bid >> 3);
}

// ---- decays of a chunk ----
// With g_r the log decay of row r, the weight of the pair (t, s), s <= t, is
// exp(g_{s+1} + .. + g_t).  It is never the quotient of two running products: those
// lose the value where one of them is small, and an infinite g (a reset) would give
// infinity less infinity.  Rows are taken in blocks of 16: across blocks the weight is
// exp(sum to the end of s's block) exp(sum of the blocks between) exp(sum within t's),
// each a sum of terms that are there; within a block the sums are formed pair by pair.
template <class T>
struct __attribute__((aligned(16))) Decays {  // (several lie one behind the other, and are read four numbers at a time)
    static constexpr int Q = kChunk<T>, B = Q / 16;
    float g[Q], in[Q], out[Q];     // of each row: log decay, weight towards the state, weight of what is read
    float head[Q], tail[Q];        // exp(sum from t's block's start to t) out_t; exp(sum behind s to its block's end) in_s
    float from[Q], to[Q];          // the same from the chunk's start, to its end
    float between[B][B];           // [i][j]: exp(sum over the blocks between j < i)
    float all, whole;              // the sum of all, and its exponential
    float most_in, most_out, grow; // largest weights; at least as much as any product of decays (float16 only)
    int odd;                       // the chunk has to be walked step by step
};
// one wave, lane r (of Q) with row r's values
template <class T>
__device__ __forceinline__ void put_decays(Decays<T>& d, float g, float in, float out, int lane) {
    constexpr int Q = kChunk<T>, B = Q / 16;
    const bool row = lane < Q;
    g = row ? g : 0.0f, in = row ? in : 0.0f, out = row ? out : 0.0f;
    const float pre = row_prefix(g), suf = row_suffix(dpp_zero<0x101>(g));
    float sum[B], before = 0.0f, after = 0.0f, all = 0.0f;
    const int block = lane >> 4;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        sum[b] = of_lane(pre, 16 * b + 15);
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
    // growth and weights that could pass the type's range in a part of a product (kHuge), NaN
    constexpr bool H = std::is_same<T, f16>::value;
    const float up = across_rows(row_sum(fmaxf(g, 0.0f))), grow = exp_f<F>(up);
    const bool odd = !(up < (H ? 4.0f : 40.0f)) ||
                     __ballot(g != g || !(fabsf(in) * grow < 0x1p60f) || !(fabsf(out) < 0x1p14f));
    if (lane == 0) {
        d.all = all, d.whole = exp_f<F>(all);
        d.odd = odd;
        if (H) d.grow = grow;
    }
    if constexpr (H) {
        float a = fabsf(in), b = fabsf(out);
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) a = fmaxf(a, __shfl_xor(a, k)), b = fmaxf(b, __shfl_xor(b, k));
        if (lane == 0) d.most_in = a, d.most_out = b;
    }
}
// The weights out_t E in_s of the lane's elements of tile (ti, si): t = 16 ti + (lane & 15),
// s = 16 si + 4 (lane >> 4) + i.  Across blocks:
template <class T>
__device__ __forceinline__ f32x4 weights_across(const Decays<T>& d, int ti, int si, int lane) {
    const float h = d.head[16 * ti + (lane & 15)] * d.between[ti][si];
    return *reinterpret_cast<const f32x4*>(&d.tail[16 * si + 4 * (lane >> 4)]) * h;
}
// within block ti (zero for s > t): sums of t's own four steps up to t, of s's four behind s
// (up to t where both are the same) and of the fours between
template <class T>
__device__ __forceinline__ f32x4 weights_within(const Decays<T>& d, int ti, int lane) {
    const int tl = lane & 15, gl = lane >> 4;
    const int tb = tl >> 2, tr = tl & 3;
    const bool same = tb == gl;
    const f32x4 q1 = *reinterpret_cast<const f32x4*>(&d.g[16 * ti + 4]);
    const f32x4 q2 = *reinterpret_cast<const f32x4*>(&d.g[16 * ti + 8]);
    const f32x4 qt = *reinterpret_cast<const f32x4*>(&d.g[16 * ti + 4 * tb]);
    f32x4 qs = *reinterpret_cast<const f32x4*>(&d.g[16 * ti + 4 * gl]);
    float rest = qt[0] + (tr > 0 ? qt[1] : 0.0f) + (tr > 1 ? qt[2] : 0.0f) + (tr > 2 ? qt[3] : 0.0f);
    rest += gl < 1 && tb > 1 ? (q1[0] + q1[1]) + (q1[2] + q1[3]) : 0.0f;
    rest += gl < 2 && tb > 2 ? (q2[0] + q2[1]) + (q2[2] + q2[3]) : 0.0f;
    rest = same ? 0.0f : rest;
#pragma unroll
    for (int i = 1; i < 4; ++i) qs[i] = same && i > tr ? 0.0f : qs[i];
    const float e[4] = {rest + (qs[1] + (qs[2] + qs[3])), rest + (qs[2] + qs[3]), rest + qs[3], rest};
    const float o = d.out[16 * ti + tl];
    const f32x4 w = *reinterpret_cast<const f32x4*>(&d.in[16 * ti + 4 * gl]);
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = 4 * gl + i <= tl ? exp_f<kFine<T>>(e[i]) * (o * w[i]) : 0.0f;
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
    Source key, query, value;
    bool fast;                        // all three vectors of columns, and results stored four values at once
    View4 result;                     // result.data null: the states alone
    View3 g, beta;                    // float; beta.data nullable
    float scale;
    const float* D;                   // [H] nullable
    const float* x_in;                // [states, H, N, P] nullable
    float* x_out;                     // nullable
    float* saved;                     // nullable: the states before every chunk
    int64_t segment;                  // steps of a segment, whole chunks
    int64_t items;                    // segments of all sequences
    float* seg_x;                     // [items, H, N, P]: what a segment leaves of a state of zero (the first: of x_in)
    float* seg_decay;                 // [items, H]: the sum of a segment's log decays
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
// and the gradients of the states behind them, both as kept (below)
struct PairArgs {
    Seqs q;
    int64_t Bsz, H, G, N, P;
    float scale;
    Source qv, k, v, dy;
    bool fast;                 // all four vectors of columns
    View4 dq, dk;
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
// sequence + chunk) of [rows, H, padded N / 16, padded P, 16], zero where there is none.
// (Sixteen keys of a value lie together: the walk's lane has four of them, and stores a vector.
// A vector instead of four numbers saves it a sixteenth of its vector instructions.)
__host__ __device__ inline int64_t padded_keys(int64_t N) { return (N + 15) / 16 * 16; }
__host__ __device__ inline int64_t padded_values(int64_t P) { return (P + 31) / 32 * 32; }
__host__ __device__ inline int64_t linear_rows(int64_t S, int64_t L, bool packed, int Q) {
    return packed ? L / Q + S : S * ((L + Q - 1) / Q);
}
__device__ __forceinline__ int64_t linear_row(const Seqs& q, const Item& it, int Q) {
    return q.offsets ? (int64_t)(it.beg / Q) + it.s : (int64_t)it.s * ((q.L + Q - 1) / Q);
}

}  // namespace ssm

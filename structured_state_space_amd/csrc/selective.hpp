// Shared pieces of the selective state-space kernels: element types, the
// argument blocks the launchers take, the map from a work item to a stretch of
// one sequence, quad (4-lane) exchanges and the scalar functions.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm.h"

namespace ssm {

// ---- element types: activations are read to float32 and rounded once on the way out ----
struct bf16 { uint16_t v; };
struct f16 { _Float16 v; };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __uint_as_float((uint32_t)x.v << 16); }
__device__ __forceinline__ float to_f(f16 x) { return (float)x.v; }
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ f16 from_f<f16>(float x) { return f16{(_Float16)x}; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) {  // round to nearest, ties to even
    return bf16{__builtin_bit_cast(uint16_t, (__bf16)x)};
}

// 8 consecutive elements as one (or, in float32, two) 16-byte accesses; the
// address needs no more than the element's own alignment
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec8 {
    T v[8];
};
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec4 {
    T v[4];
};

// ---- views: element (b, h, l) at data + b sb + h sh + l sl (in elements) ----
struct View3 {
    const void* data = nullptr;
    int64_t sb = 0, sh = 0, sl = 0;
};
struct View4 {
    const void* data = nullptr;
    int64_t sb = 0, sg = 0, sn = 0, sl = 0;
};

// ---- sequences of a call ----
// dense: sequence s is batch row s, of L or lengths[s] steps.  packed (offsets
// given): one batch row of L steps, sequence s at [offsets[s], offsets[s+1]).
// Values outside [0, L] are clamped, so that no content of these arrays can
// lead an access out of the tensors.
struct Seqs {
    int64_t S = 0, L = 0;
    const int32_t* offsets = nullptr;
    const int32_t* lengths = nullptr;
    const int32_t* slots = nullptr;
    int64_t n_slots = 0;
};

// the stretch of steps a workgroup handles
struct Item {
    int s;         // sequence
    int c;         // its chunk
    int64_t row;   // batch row
    int beg, end;  // the sequence's steps along the row's time axis
    int64_t state; // its state row, or -1: no such state, nothing to do
};

__device__ __forceinline__ void seq_bounds(const Seqs& q, int s, int64_t& row, int& beg, int& end) {
    const int L = (int)q.L;
    if (q.offsets) {
        row = 0;
        beg = min(max(q.offsets[s], 0), L);
        end = min(max(q.offsets[s + 1], beg), L);
    } else {
        row = s;
        beg = 0;
        end = q.lengths ? min(max(q.lengths[s], 0), L) : L;
    }
}

__device__ __forceinline__ int chunks_of(int len, int Q) { return max(1, (int)(((int64_t)len + Q - 1) / Q)); }

// Work items enumerate the chunks of Q steps of every sequence, at least one
// per sequence.  Dense: item = s * ceil(L/Q) + c.  Packed: the sequences'
// chunks one behind the other; a wave finds its item by a prefix sum over 64
// sequences at a time.  Returns false where the item is behind the last one.
__device__ __forceinline__ bool find_item(const Seqs& q, int64_t item, int Q, Item& it) {
    if (!q.offsets) {
        const int per = chunks_of((int)q.L, Q);
        it.s = (int)(item / per);
        it.c = (int)(item % per);
    } else {
        const int lane = threadIdx.x & 63;
        int64_t left = item;
        int s0 = 0, found = -1;
        for (; s0 < q.S; s0 += 64) {
            int n = 0;
            if (s0 + lane < q.S) {
                int64_t row;
                int b, e;
                seq_bounds(q, s0 + lane, row, b, e);
                n = chunks_of(e - b, Q);
            }
            int64_t incl = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
            const uint64_t hit = __ballot(left < incl);
            if (hit) {
                found = __builtin_ctzll(hit);
                const int64_t before = __shfl(incl - n, found);
                left -= before;
                break;
            }
            left -= __shfl(incl, 63);
        }
        if (found < 0) return false;
        it.s = s0 + found;
        it.c = (int)left;
    }
    it.s = __builtin_amdgcn_readfirstlane(it.s);
    it.c = __builtin_amdgcn_readfirstlane(it.c);
    seq_bounds(q, it.s, it.row, it.beg, it.end);
    it.state = it.s;
    if (q.slots) {
        const int64_t slot = q.slots[it.s];
        it.state = slot >= 0 && slot < q.n_slots ? slot : -1;
    }
    return true;
}

// items a launch has to cover (host side): exact when dense, an upper bound when packed
inline int64_t item_count(const Seqs& q, int64_t Q) {
    if (!q.offsets) return q.S * ((q.L + Q - 1) / Q);
    return q.S + q.L / Q;
}

// a launch has less than 2^32 threads in all
inline bool grid_fits(int64_t wgs, int threads) { return wgs < ((int64_t)1 << 32) / threads; }

// Steps of a chunk, a multiple of kTile, for `blocks` workgroups along the
// channels; q.L or more: no chunks.  Chunks cost a launch over nearly all of the
// steps more (0.65 of the forward pass, 0.25 of the backward), so they are made
// where 512 workgroups come out of `least` chunks or more.
// Measured at 1024 channels (16 workgroups a row), N = 16, 4096 steps bf16, forward:
// 8 rows 337 us whole, 249 in 4 chunks; 10 rows 337 and 311 in 3; 12 rows 338 and
// 454 in 2.  Both directions, 2048 steps: 9 rows 738 whole and 669 with the backward
// pass in 3, 12 rows 720 and 859 in 2.
// N = 64 forward, whose workgroups have a CU to themselves: 8 rows 422 and 380 in 4,
// 10 rows 422 and 502 in 3.
// The backward pass's second launch has one workgroup to a CU and takes 512 in two
// rounds.  256 in its place, N = 16, that pass alone: 9 rows of 1024 x 2048 545 us
// against 468 with 512, 1 x 2048 x 8192 375 and 355, 4 rows of 1024 x 2048 191 and 187;
// but 1 x 256 x 16384 124 and 149.
// A chunk has four tiles where 256 workgroups come out of that (256 channels in 2
// groups, N = 64, 8 rows x 1024 steps: 74 us against 87 with two tiles), else two
// at least (256 channels, N = 64, 1 row x 2048 steps: 49 us against 66 with four;
// but 64 channels, N = 16, x 16384: 87 and 60).
// Packed sequences count as one long one: the host does not know their lengths.  4096
// steps forward, N = 16, whole and in chunks, of one sequence, two (2100 and 1996)
// and eight of 512: 8192 channels in 4 chunks 340 and 238, 183 and 245, 146 and 151 us;
// 10240 channels in 3 342 and 313, 279 and 313, 194 and 188; 12288 in 2 341 and 387,
// 280 and 392, 225 and 233.
constexpr int kTile = 32;
inline int64_t chunk_steps(const Seqs& q, int64_t blocks, int least) {
    const int64_t total = blocks * (q.offsets ? 1 : q.S), chunks = 512 / total;
    int64_t Q = q.L;
    if (chunks >= least) {
        Q = (q.L + chunks - 1) / chunks;
        const int64_t few = q.L / (4 * kTile) * total >= 256 ? 4 * kTile : 2 * kTile;
        if (Q < few) Q = few;
    }
    Q = (Q + kTile - 1) / kTile * kTile;
    return Q < ((int64_t)1 << 30) ? Q : (int64_t)1 << 30;
}

// ---- a workgroup of the scan kernels ----
// 64 channels of one group, 32 steps to a tile, 512 threads in two roles.
// Moving a tile: thread by thread four elements of every activation, in vector
// accesses along whichever axis is contiguous; they turn delta into dt and hand
// the steps' values to the other role, and take its results back, through LDS.
// Running a tile: eight neighbouring lanes per channel, lane p the S states
// n = p S + j; a wave has 8 channels.  (Lanes that loaded their own channel's steps
// made 28 cache accesses per 64-lane load where the vectors make 8.)
constexpr int kChannels = 64;
constexpr int kScanThreads = kChannels * 8;
constexpr int kOwn = 4;

enum Order {
    kRows,    // steps contiguous: a thread moves four steps of one channel
    kTokens,  // channels contiguous: four channels of one step
    kAny,     // neither: the same, element by element
};

struct Place {
    int tid, p, wave, c, g, blk, h;  // c, h: the running lane's channel in the block and of all (clamped)
    int valid;                       // channels of the block
    int64_t first;                   // the block's first channel
    bool live;                       // the running lane's channel exists
};
__device__ __forceinline__ Place place_of(int cb, int per_group, int64_t H, int64_t G) {
    Place l;
    l.tid = threadIdx.x;
    l.p = l.tid & 7;
    l.wave = __builtin_amdgcn_readfirstlane(l.tid >> 6);
    l.g = cb / per_group;
    l.blk = cb % per_group;
    const int Hg = (int)(H / G);
    l.first = (int64_t)l.g * Hg + l.blk * kChannels;
    l.valid = min(kChannels, Hg - l.blk * kChannels);
    l.c = l.tid >> 3;
    l.live = l.c < l.valid;
    l.h = (int)l.first + min(l.c, l.valid - 1);
    return l;
}

// the four elements a thread moves: steps t + (kRows ? i : 0), channels
// c + (kRows ? 0 : i) of the block.  With kTokens a vector that would end behind the
// last channel is moved back to end with it (c may be negative in a block of fewer
// than four; a group has at least four), so that some elements are moved twice.
// A tensor is addressed by a base that is the same in the whole workgroup and
// moves from tile to tile, and a 32-bit distance in bytes per thread, which the
// strides' limits keep below 2^32.  (Pointers per thread took twice the registers;
// the backward pass then kept some in scratch memory, and waiting for those loads
// meant waiting for the next tile's.)
template <Order O>
struct Mover {
    int t, c, low, most;
    __device__ __forceinline__ Mover(int tid, int valid) {
        t = O == kRows ? (tid & 7) * 4 : tid >> 4;
        c = O == kRows ? tid >> 3 : (tid & 15) * 4;
        low = O == kTokens ? min(0, valid - 4) : 0;
        if (O == kTokens) c = min(c, valid - 4);
        most = O == kAny ? min(kOwn - 1, max(0, valid - 1 - c)) : kOwn - 1;
        cc = O == kTokens ? c - low : min(c, valid - 1);
    }
    __device__ __forceinline__ int step(int i) const { return t + (O == kRows ? i : 0); }
    __device__ __forceinline__ int channel(int i) const { return c + (O == kRows ? 0 : i); }
    __device__ __forceinline__ bool has(int i, int valid) const {
        return channel(i) >= 0 && channel(i) < valid;
    }
    template <class T>
    __device__ __forceinline__ char* base(const View3& v, int64_t row, const Place& l, int64_t step0) const {
        return (char*)v.data + (row * v.sb + (l.first + low) * v.sh + step0 * v.sl) * (int64_t)sizeof(T);
    }
    template <class T>
    __device__ __forceinline__ uint32_t offset(const View3& v) const {
        return ((uint32_t)cc * (uint32_t)v.sh + (uint32_t)t * (uint32_t)v.sl) * (uint32_t)sizeof(T);
    }
    template <class T>
    __device__ __forceinline__ void load(T (&r)[kOwn], const char* p, uint32_t off, const View3& v) const {
        if constexpr (O == kAny) {  // channels behind the last one read it again
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                r[i] = *reinterpret_cast<const T*>(p + (off + min(i, most) * (uint32_t)v.sh * (uint32_t)sizeof(T)));
        } else {
            const Vec4<T> w = *reinterpret_cast<const Vec4<T>*>(p + off);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) r[i] = w.v[i];
        }
    }
    // where only the tile's first nt steps exist
    template <class T>
    __device__ __forceinline__ void load_part(T (&r)[kOwn], const char* p, uint32_t off, const View3& v, int nt) const {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const uint32_t d = O == kRows ? i * (uint32_t)sizeof(T) : min(i, most) * (uint32_t)v.sh * (uint32_t)sizeof(T);
            r[i] = step(i) < nt ? *reinterpret_cast<const T*>(p + (off + d)) : from_f<T>(0.0f);
        }
    }
    template <class T>
    __device__ __forceinline__ void store(const float (&r)[kOwn], char* p, uint32_t off, const View3& v, int valid,
                                          int nt) const {
        if (O != kAny && step(O == kRows ? kOwn - 1 : 0) < nt && (O == kTokens ? c >= 0 : c < valid)) {
            Vec4<T> w;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) w.v[i] = from_f<T>(r[i]);
            *reinterpret_cast<Vec4<T>*>(p + off) = w;
        } else {
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                if (step(i) < nt && has(i, valid))
                    *reinterpret_cast<T*>(p + (off + i * (O == kRows ? 1u : (uint32_t)v.sh) * (uint32_t)sizeof(T))) =
                        from_f<T>(r[i]);
        }
    }

  private:
    int cc;
};

// the thread's number, opaque to the compiler: what is worked out from it is worked
// out here, and not kept in registers from elsewhere
__device__ __forceinline__ int anew(int tid) {
    asm volatile("" : "+v"(tid));
    return tid;
}

// a kernel's first argument, read anew from where a launch leaves its arguments:
// what a tile needs of it once is loaded then (scalar loads that hit their cache).
// Kept in scalar registers it would spill, to be read back lane by lane from a
// vector register, an instruction for each.
template <class A>
__device__ __forceinline__ A arguments() {
    using Words = const __attribute__((address_space(4))) uint64_t*;
    static_assert(sizeof(A) % 8 == 0, "whole words");
    Words p = (Words)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    uint64_t w[sizeof(A) / 8];
#pragma unroll
    for (size_t i = 0; i < sizeof(A) / 8; ++i) w[i] = p[i];
    A a;
    __builtin_memcpy(&a, w, sizeof(A));
    return a;
}

// B and C of a tile on their way to LDS in float32: row t holds, per pair k of a
// lane's states, the eight lanes' {B, B, C, C}; a thread brings K elements of either
template <class T, int S>
struct Stage {
    static constexpr int K = kTile * 8 * S / kScanThreads;  // 1, 2 or 4
    static constexpr int kRow = 16 * S + 4;                 // floats of a row (padded)
    uint32_t bo[K], co[K];  // distances from the tile's first step in bytes
    int N, tid;
    bool by_time;  // consecutive threads along B's contiguous axis
    __device__ __forceinline__ Stage(const View4& B, const View4& C, int states, int thread)
        : N(states), tid(thread), by_time(B.sl == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int t, n;
            place(k, t, n);
            bo[k] = distance(B, t, n), co[k] = distance(C, t, n);
        }
    }
    __device__ __forceinline__ void place(int k, int& t, int& n) const {
        const int e = tid + kScanThreads * k;
        t = by_time ? e % kTile : e / (8 * S);
        n = by_time ? e / kTile : e % (8 * S);
    }
    __device__ __forceinline__ uint32_t distance(const View4& v, int t, int n) const {  // padded states read the last one
        return ((uint32_t)t * (uint32_t)v.sl + (uint32_t)min(n, N - 1) * (uint32_t)v.sn) * (uint32_t)sizeof(T);
    }
    template <bool WB, bool WC>
    __device__ __forceinline__ void load(T (&b)[K], T (&c)[K], const char* Bp, const char* Cp) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (WB) b[k] = *reinterpret_cast<const T*>(Bp + bo[k]);
            if (WC) c[k] = *reinterpret_cast<const T*>(Cp + co[k]);
        }
    }
    // where only the tile's first nt steps exist: the others read the last one
    template <bool WB, bool WC>
    __device__ __forceinline__ void load_part(T (&b)[K], T (&c)[K], const View4& B, const View4& C, const char* Bp,
                                              const char* Cp, int nt) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int t, n;
            place(k, t, n);
            t = min(t, nt - 1);
            if (WB) b[k] = *reinterpret_cast<const T*>(Bp + distance(B, t, n));
            if (WC) c[k] = *reinterpret_cast<const T*>(Cp + distance(C, t, n));
        }
    }
    // padded states, and steps behind the last one, become zero
    template <bool WB, bool WC>
    __device__ __forceinline__ void store(const T (&b)[K], const T (&c)[K], float* to, int nt) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int t, n;
            place(k, t, n);
            float* at = to + t * kRow + ((n % S / 2) * 8 + n / S) * 4 + (n & 1);
            const bool in = t < nt && n < N;
            if (WB) at[0] = in ? to_f(b[k]) : 0.0f;
            if (WC) at[2] = in ? to_f(c[k]) : 0.0f;
        }
    }
};
// the base of B or C in a tile
template <class T>
__device__ __forceinline__ const char* group_base(const View4& v, int64_t row, int g, int64_t step0) {
    return (const char*)v.data + (row * v.sb + g * v.sg + step0 * v.sl) * (int64_t)sizeof(T);
}

// lane exchanges (v_*_dpp)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
// lane q of a quad gets the sum over the quad of p_q: 9 instructions for four sums
__device__ __forceinline__ float quad_sums(float p0, float p1, float p2, float p3, bool odd, bool high) {
    const float a = (odd ? p1 : p0) + dpp<0xB1>(odd ? p0 : p1);
    const float b = (odd ? p3 : p2) + dpp<0xB1>(odd ? p2 : p3);
    return (high ? b : a) + dpp<0x4E>(high ? a : b);
}
// Pairs of floats per step and channel in LDS: {dt, dt u} on the way to the
// running lanes, the two quads' sums over a channel's states on the way back.
// Four floats of room behind every eighth channel and the row's length keep both
// roles' accesses (16 bytes of two channels at a time, 16 threads per step; eight
// bytes of eight channels; four bytes of four steps) off each other's banks.
constexpr int kPairRow = 176;
__device__ __forceinline__ int pair_at(int c) { return c * 2 + (c >> 3) * 4; }
// lane p leaves its quad's sum of step 4 g + (p & 3); the mover adds the two quads'
__device__ __forceinline__ void put_sums(float* to, int g, float s, int c, int p, bool add = false) {
    float* at = to + (4 * g + (p & 3)) * kPairRow + pair_at(c) + (p >> 2);
    *at = add ? *at + s : s;
}
template <Order O>
__device__ __forceinline__ void get_sums(float (&r)[kOwn], const float* from, const Mover<O>& m) {
    if (O == kTokens && m.c >= 0 && (m.c & 3) == 0) {
        const float4* v = reinterpret_cast<const float4*>(from + m.t * kPairRow + pair_at(m.c));
        const float4 x = v[0], y = v[1];
        r[0] = x.x + x.y, r[1] = x.z + x.w, r[2] = y.x + y.y, r[3] = y.z + y.w;
    } else {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const float2 v = *reinterpret_cast<const float2*>(from + m.step(i) * kPairRow + pair_at(max(m.channel(i), 0)));
            r[i] = v.x + v.y;
        }
    }
}
template <Order O>
__device__ __forceinline__ void put_pairs(float* to, const float (&x)[kOwn], const float (&y)[kOwn], const Mover<O>& m,
                                          int valid) {
    if (O == kTokens && m.c >= 0 && (m.c & 3) == 0) {
        float4* v = reinterpret_cast<float4*>(to + m.t * kPairRow + pair_at(m.c));
        v[0] = make_float4(x[0], y[0], x[1], y[1]);
        v[1] = make_float4(x[2], y[2], x[3], y[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (m.has(i, valid))
                *reinterpret_cast<float2*>(to + m.step(i) * kPairRow + pair_at(m.channel(i))) = make_float2(x[i], y[i]);
    }
}
// a lane's S states of a row [Np] of a workspace
template <int S>
__device__ __forceinline__ void load_states(float (&r)[S], const float* p) {
#pragma unroll
    for (int k = 0; k < S; k += 2) {
        const float2 v = *reinterpret_cast<const float2*>(p + k);
        r[k] = v.x, r[k + 1] = v.y;
    }
}
template <int S>
__device__ __forceinline__ void store_states(const float (&r)[S], float* p) {
#pragma unroll
    for (int k = 0; k < S; k += 2) *reinterpret_cast<float2*>(p + k) = make_float2(r[k], r[k + 1]);
}

// how the activations of a call lie, from their views (null ones aside)
inline Order order_of(const View3* const* v, int n, int64_t per_group) {
    bool rows = true, tokens = per_group >= 4;
    for (int i = 0; i < n; ++i) {
        if (!v[i]->data) continue;
        rows = rows && v[i]->sl == 1;
        tokens = tokens && v[i]->sh == 1;
    }
    return rows ? kRows : tokens ? kTokens : kAny;
}

// ---- scalar functions ----
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = 1.925963033500717e-08f;  // log2(e) - kLog2e
constexpr float kLn2 = 0.6931471805599453f;

// exp(v).  FINE: to about one unit in the last place up to |v| = 80, the product
// v log2(e) in two parts; else, and beyond 80 (where only results below 2e-35 or
// their reciprocals show it), its rounding costs |v| / 2 units more, for six
// instructions fewer.
// Kernels take FINE for float32 activations; 16-bit ones are coarser by 2^13.
template <bool FINE>
__device__ __forceinline__ float exp_f(float v) {
    const float p = v * kLog2e;
    const float e = __builtin_amdgcn_exp2f(p);
    if (!FINE) return e;
    const float lo = fmaf(v, kLog2eLo, fmaf(v, kLog2e, -p));
    // far from 0, where e may be infinite or lo NaN, exp2 alone
    return fabsf(v) < 80.0f ? fmaf(e, lo * kLn2, e) : e;
}

// log(1 + exp(v)); above 20 it is v to float32.  log1p(e) = log(w) + (e - (w - 1))/w
// with w = fl(1 + e); where e >= 1 the second term, up to one unit of the result, is
// left out, elsewhere w stands for 1 in it (up to 0.9 units, at e near 0.6).  With
// exact exp and log the result is within 3.1 units.  `slope` is e / (1 + e).
template <bool FINE, bool SLOPE = false>
__device__ __forceinline__ float softplus_f(float v, float* slope = nullptr) {
    const float e = exp_f<FINE>(v);
    const float w = 1.0f + e;
    const float c = e < 1.0f ? e - (w - 1.0f) : 0.0f;
    const float r = fmaf(__builtin_amdgcn_logf(w), kLn2, c);
    if (SLOPE) *slope = v > 20.0f ? 1.0f : e * __builtin_amdgcn_rcpf(w);
    return v > 20.0f ? v : r;
}

template <bool FINE>
__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.0f + exp_f<FINE>(-v));
}
template <bool FINE>
__device__ __forceinline__ float silu_f(float v) {
    return v * sigmoid_f<FINE>(v);
}
template <class T>
constexpr bool kFine = sizeof(T) == 4;

// x <- x exp2(s A2) + e: states (or gradients) over a chunk whose steps add up to s and
// which ends in e from zero.  The sum may pass float32 where no step does (with an A of
// 0 the factor stays 1), and so may the factor where x is zero, small or infinite: x
// takes its square root twice, which is held finite and above zero.  (Factors beyond
// 2^254 or below 2^-252 are cut there: normal x become infinite, or less than 2^-123.)
template <int S>
__device__ __forceinline__ void over_chunk(float (&x)[S], float s, const float (&A2)[S], const float (&e)[S]) {
    constexpr float kMost = 3.402823466e38f;
    const float half = 0.5f * __builtin_amdgcn_fmed3f(s, -kMost, kMost);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const float root = __builtin_amdgcn_exp2f(__builtin_amdgcn_fmed3f(half * A2[j], -126.0f, 127.0f));
        x[j] = fmaf(x[j] * root, root, e[j]);
    }
}

// ---- argument blocks ----
struct ScanArgs {
    Seqs q;
    int64_t Bsz, H, N, G;
    int softplus;
    View3 u, delta, z, y;  // z.data, y.data nullable
    View4 B, C;
    const float* A;
    const float* D;           // nullable
    const float* delta_bias;  // nullable
    const float* x_in;        // [states, H, N] nullable
    float* x_out;             // nullable
    float* saved;             // nullable: states every kSaveSteps steps, for the backward pass
};

struct ScanGradArgs {
    ScanArgs f;      // the forward call's arguments (y, x_out, saved unused)
    const float* saved;
    View3 dy;
    View3 du, ddelta, dz;
    View4 dB, dC;
    float *dA, *dD, *ddelta_bias;  // dD, ddelta_bias nullable
    const float* dx_out;           // gradient of the final states, nullable
    float* dx_in;                  // gradient of the initial states, nullable
};

struct ConvArgs {
    Seqs q;
    int64_t H;
    int width, silu;
    View3 u, y;
    const float* weight;   // [H, width]
    const float* bias;     // [H] nullable
    const void* state_in;  // [states, H, width - 1] of u's type, oldest first; nullable
    void* state_out;       // nullable, may be state_in
};

struct ConvGradArgs {
    ConvArgs f;  // the forward call's arguments (y, state_out unused; states are per sequence)
    View3 dy, du;
    float *dweight, *dbias;    // nullable
    const float* dstate_out;   // [S, H, width - 1], nullable
    float* dstate_in;          // nullable
};

struct StepArgs {
    int64_t Bsz, H, N, G;
    int softplus;
    const int32_t* slots;  // nullable
    int64_t n_slots;
    const void *u, *delta, *z, *B, *C;  // [Bsz, H], [Bsz, G, N]; strides of rows (groups, states) below
    void* y;
    int64_t u_row, delta_row, z_row, y_row, B_row, B_group, B_state, C_row, C_group, C_state;
    const float *A, *D, *delta_bias;
    float* x;  // [states, H, N], updated
};

struct ConvStepArgs {
    int64_t Bsz, H;
    int width, silu;
    const int32_t* slots;
    int64_t n_slots;
    const void* u;
    void* y;
    int64_t u_row, y_row;
    const float *weight, *bias;
    void* state;  // [states, H, width - 1], updated
};

// states per channel as the kernels hold them: 2, 4 or 8 on each of its lanes
__host__ __device__ inline int64_t padded_states(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : 64; }

// steps between two saved states, and where they lie: sequence s keeps its
// k-th at row saved_row + k of [rows, H, padded_states(N)]
constexpr int kSaveSteps = kTile;
__host__ __device__ inline int64_t saved_rows(int64_t S, int64_t L, bool packed) {
    return packed ? L / kSaveSteps + S : S * ((L + kSaveSteps - 1) / kSaveSteps);
}
__device__ __forceinline__ int64_t saved_row(const Seqs& q, const Item& it) {
    return q.offsets ? (int64_t)(it.beg / kSaveSteps) + it.s
                     : (int64_t)it.s * ((q.L + kSaveSteps - 1) / kSaveSteps);
}

}  // namespace ssm

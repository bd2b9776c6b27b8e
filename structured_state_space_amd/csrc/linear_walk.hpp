// The walk over the chunks of a sequence, for linear attention forwards and for the
// gradient of its values backwards (include/ssm.h: ssm_linear_attention).
#pragma once

#include "linear.hpp"

namespace ssm {

constexpr int kWalkThreads = 512;
constexpr int kWalkWaves = kWalkThreads / 64;
constexpr int kWalkValues = 64;  // values of a workgroup

// A workgroup has one head, 64 of its values and one segment of a sequence, and takes a
// chunk of rows at a time.  With the pairs' weights M_ts = out_t (q_t . k_s) E_ts in_s
// (s <= t) the chunk's results are
//   result_t = sum_s M_ts value_s + out_t E_t x^T q_t + D value_t,
// and the state becomes E x + sum_s E'_s in_s k_s value_s^T: four matrix products.  The state
// stays in float32 in registers, as the matrix instruction leaves it: a wave has 16 values and
// half of the keys, and of the results those values and half of the steps.  The registers are
// operands as they are: a wave multiplies its keys with all steps, and either half gives the other
// its steps' results through LDS once a chunk.  (The rounded state itself there, of all keys for
// half of the steps, takes twice the room in two parts, and a unit then one workgroup instead of
// two.)  M goes through LDS, a tile of 16 x 16 pairs from a wave.
// 256 heads of 2048 steps, 128 keys and 64 values, bf16, with the states saved: 163 us, two waves to
// a SIMD that issue vector instructions in half of the cycles (570 a wave and chunk, a quarter of
// them for the splits) and wait for each other, three barriers to a chunk.  (Four waves with all
// keys and steps of their values needed no exchange of the state, but waited more; two sets of tiles
// and two barriers were no faster: with M and the state in one part 265 us instead of 153, and forwards
// 240 heads of 8192 steps 523 us instead of 447.)
// M and the state are operands in two parts of 16 bits (kShort), what is added to the state in
// kParts, and D value stays in float32: the results have the error of their own rounding.  (In one
// part: 1.4 times that, for 6% less time over 16384 steps of 32 heads and 5% over 4 x 2048 steps of 64
// with their gradients.)
// ENDS: the first of two passes, which finds each segment's end state for the second.
// OUT: results wanted.  FAST: the tensors' usual layout (WalkArgs), in a kernel without the code for
// others: 5800 instructions instead of 8100, and addresses that do not fill the registers.
template <class T, int NP, bool OUT, bool REVERSE, bool ENDS, bool FAST>
__global__ __launch_bounds__(kWalkThreads, NP * sizeof(T) > 256 ? 2 : 4) void linear_walk_kernel(const WalkArgs a) {
    constexpr int Q = kChunk<T>, TT = Q / 16, HT = TT / 2, KK = NP / 32, SS = Q / 32, NT = NP / 32;  // NT: of a wave
    constexpr int KS = NP + kRoom<T>, VS = kWalkValues + kRoom<T>, K2 = kShort<T>;
    using Pairs = PairPlaces<T>;
    constexpr bool F16 = std::is_same<T, f16>::value;
    struct __attribute__((aligned(16))) Shared {
        T k[Q * KS];
        T v[Q * VS];
        T q[OUT ? Q * KS : 8];
        T m[OUT ? K2 * Pairs::kSize : 8];
        union {
            f32x4 across[OUT ? kWalkWaves : 1][HT][64];  // for each wave, what its other keys' wave has for it
            float sums[2][2][kWalkValues];
        };
        Decays<T> d[2];
        uint32_t most[3][kWalkWaves];
        float most_x[kWalkWaves];
        int odd[kWalkWaves];
    };
    __shared__ Shared sh;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pq = wave & 3, half = wave >> 2;
    const int blocks = (int)((a.P + kWalkValues - 1) / kWalkValues);
    const int pb = (int)(blockIdx.x % blocks), h = (int)(blockIdx.x / blocks % (int)a.H);
    const int64_t item = (int64_t)(blockIdx.x / blocks) / a.H;
    Item it;
    if (!find_item(a.q, item, (int)a.segment, it) || it.state < 0) return;
    const int len = it.end - it.beg, segments = chunks_of(len, (int)a.segment);
    // (descending offsets make more segments than there are items: a sequence without all of its own is left out)
    if (it.c >= segments || item - it.c + segments > a.items) return;
    if (ENDS && segments == 1) return;
    const int pos = REVERSE ? segments - 1 - it.c : it.c;  // in the order of the walk
    const int chunks = (len + Q - 1) / Q, per = (int)(a.segment / Q);
    const int c0 = it.c * per, c1 = min(c0 + per, chunks);

    const int N = (int)a.N, P = (int)a.P;
    const int p0 = pb * kWalkValues;
    const bool live = p0 + 16 * pq < P;
    // the wave's tiles of rows: of four the first and last or the two between, as many pairs in either
    auto tile_of = [](int half, int t) { return HT == 2 && t ? 3 - half : half; };
    auto tile = [&](int t) { return tile_of(half, t); };
    f32x4 x[NT];
    // the lane's states of a row of a [rows, H, N, P] array: n = 16 (NT half + tile) + 4 gl + i, value p
    auto exchange = [&](f32x4 (&x)[NT], auto* base, int64_t r, auto&& each) {
        const int lane = anew(threadIdx.x) & 63, p = p0 + 16 * pq + (lane & 15), n0 = 16 * NT * half + 4 * (lane >> 4);
        auto* at = base + ((r * a.H + h) * N + n0) * P + p;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = each(x[n][i], at + (16 * n + i) * P, n0 + 16 * n + i < N && p < P);
    };
    auto get = [&](const float* base, int64_t r) {
        exchange(x, base, r, [](float, const float* at, bool there) { return there ? *at : 0.0f; });
    };
    auto put = [&](float* base, int64_t r, float factor) {
        exchange(x, base, r, [=](float v, float* at, bool there) {
            if (there) *at = v * factor;
            return v;
        });
    };
    const int grp = h / (int)(a.H / a.G);
    // the next chunk's first step
    const int first = it.beg + (REVERSE ? c1 - 1 : c0) * Q;
    const char* key = a.key.data + it.row * a.key.sb + grp * a.key.sg + first * a.key.sl;
    const char* query = a.query.data + it.row * a.query.sb + grp * a.query.sg + first * a.query.sl;
    const char* value = a.value.data + it.row * a.value.sb + h * a.value.sg + p0 * a.value.sn + first * a.value.sl;
    T* result = (T*)a.result.data + it.row * a.result.sb + h * a.result.sg + (int64_t)(p0 + 16 * pq) * a.result.sn + first * a.result.sl;
    const float* gs = (const float*)a.g.data + it.row * a.g.sb + h * a.g.sh;
    const float* bs = a.beta.data ? (const float*)a.beta.data + it.row * a.beta.sb + h * a.beta.sh : nullptr;
    const float skip = a.D ? a.D[h] : 0.0f;
    const bool vectors = FAST || (a.result.sn == 1 && P % 4 == 0);  // four values are stored at once
    const int Np = (int)padded_keys(a.N), Pp = (int)padded_values(a.P);
    float* saved = a.saved && !ENDS ? a.saved + (linear_row(a.q, it, Q) * a.H + h) * Np * Pp : nullptr;

    const int count = c1 - c0;
    auto chunk = [&](int k) { return REVERSE ? c1 - 1 - k : c0 + k; };
    Carrier<T, NP, kWalkThreads, FAST> ck, cq;
    Carrier<T, kWalkValues, kWalkThreads, FAST> cv;
    auto load = [&](int k) {
        const int nt = min(Q, it.end - it.beg - chunk(k) * Q), tid = threadIdx.x;
        ck.load(key, a.key, N, nt, tid);
        cv.load(value, a.value, P - p0, nt, tid);
        if (OUT) cq.load(query, a.query, N, nt, tid);
        constexpr int64_t D = REVERSE ? -Q : Q;
        key += D * a.key.sl, value += D * a.value.sl, query += D * a.query.sl;
    };
    // The decays are worked out a chunk ahead by the last wave, from what it loaded a chunk before.
    float g = 0.0f, in = 0.0f, out = 0.0f;
    auto load_decays = [&](int k) {
        const int lane = threadIdx.x & 63, t0 = it.beg + chunk(k) * Q, o = REVERSE ? Q - 1 - lane : lane, t = t0 + o;
        g = in = out = 0.0f;
        if (lane < Q && t < it.end) {
            const float b = bs ? bs[t * a.beta.sl] : 1.0f;
            const int tg = REVERSE ? t + 1 : t;
            g = tg < it.end ? gs[tg * a.g.sl] : 0.0f;
            in = REVERSE ? a.scale : b;
            out = REVERSE ? b : a.scale;
        }
    };
    auto most_state = [&]() {  // float16: the largest finite magnitude of the wave's states
        float m = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = fabsf(x[n][i]);
                m = fmaxf(m, v < INFINITY ? v : 0.0f);
            }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        if ((threadIdx.x & 63) == 0) sh.most_x[wave] = m;
    };
    if (count > 0) {
        load(0);
        if (wave == kWalkWaves - 1) load_decays(0);
    }
    // the state, while the first chunk's loads are under way
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = f32x4{0, 0, 0, 0};
    // the item of the segment at a place of the walk
    auto item_at = [&](int j) { return item - it.c + (REVERSE ? segments - 1 - j : j); };
    double decay = 0.0;  // its logarithm, of the segment
    if (ENDS) {
        if (pos == 0 || pos == segments - 1) {
            // the last one's end is not needed: its place keeps the initial state, which the
            // final state may overwrite while the second pass still needs it
            if (a.x_in) get(a.x_in, it.state);
            if (pos != 0) {
                put(a.seg_x, item, 1.0f);
                return;
            }
        }
    } else if (segments == 1) {
        if (a.x_in) get(a.x_in, it.state);
    } else {
        get(a.seg_x, item_at(pos == 0 ? segments - 1 : 0));
        // the segments between, several under way.  A segment's decay is the exponential of the sum of
        // its logarithms, taken twice by halves: a product of its chunks' decays could pass float32 on
        // the way to a number, and what is zero stays zero beside one that does.
        constexpr int A = NT > 4 ? 2 : 4;
        for (int j = 1; j < pos; j += A) {
            f32x4 y[A][NT];
            float e[A];
#pragma unroll
            for (int i = 0; i < A; ++i) {
                const int64_t before = item_at(min(j + i, pos - 1));
                e[i] = exp_f<kFine<T>>(0.5f * a.seg_decay[before * a.H + h]);
                exchange(y[i], a.seg_x, before, [](float, const float* at, bool there) { return there ? *at : 0.0f; });
            }
#pragma unroll
            for (int i = 0; i < A; ++i)
                if (j + i < pos) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            x[n][r] = x[n][r] == 0.0f ? y[i][n][r] : fmaf(x[n][r] * e[i], e[i], y[i][n][r]);
                }
        }
    }

    if (count > 0) {
        if (wave == kWalkWaves - 1) {
            put_decays<T>(sh.d[0], g, in, out, threadIdx.x & 63);
            if (count > 1) load_decays(1);
        }
        if (OUT) {
            if (F16) most_state();
            // pairs s > t within two blocks of a product stay zero
            for (int i = threadIdx.x; i < K2 * Pairs::kSize; i += kWalkThreads) sh.m[i] = from_f<T>(0.0f);
        }
    }
    for (int k = 0; k < count; ++k) {
        const int c = chunk(k), t0 = it.beg + c * Q, nt = min(Q, it.end - t0);
        const int tid = anew(threadIdx.x), lane = tid & 63, tl = lane & 15, gl = lane >> 4;  // (addresses are not kept)
        const Decays<T>& d = sh.d[k & 1];
        if (saved && p0 + 16 * pq < Pp) {
            float* at = saved + (int64_t)c * a.H * Np * Pp + (NT * half * Pp + p0 + 16 * pq + tl) * 16 + 4 * gl;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (16 * (NT * half + n) < Np) *reinterpret_cast<f32x4*>(at + 16 * n * Pp) = x[n];
        }
        __syncthreads();  // the last chunk's tiles have been read
        ck.clear(a.key.lay, N, nt, tid);
        cv.clear(a.value.lay, P - p0, nt, tid);
        ck.template store<REVERSE>(sh.k, a.key.lay, tid);
        cv.template store<REVERSE>(sh.v, a.value.lay, tid);
        float sx = 1.0f;
        Frag<T> state[OUT ? (NT + 1) / 2 : 1][K2];
        if (OUT) {
            cq.clear(a.query.lay, N, nt, tid);
            cq.template store<REVERSE>(sh.q, a.query.lay, tid);
            if (F16) sx = to_range<T>(fmaxf(sh.most_x[pq], sh.most_x[pq + 4]));
            // the state's registers are operands as they are, of the wave's half of the keys
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = i < 4 ? x[n][i] * sx : NT > 1 ? x[n + (NT > 1)][i - 4] * sx : 0.0f;
                split<T>(u, state[n / 2]);
            }
        }
        {
            uint32_t mk = ck.most(), mv = cv.most(), mq = OUT ? cq.most() : 0;
            if constexpr (F16) {
#pragma unroll
                for (int i = 1; i < 64; i <<= 1) {
                    mk = max(mk, (uint32_t)__shfl_xor((int)mk, i)), mv = max(mv, (uint32_t)__shfl_xor((int)mv, i));
                    if (OUT) mq = max(mq, (uint32_t)__shfl_xor((int)mq, i));
                }
                if (lane == 0) sh.most[0][wave] = mk, sh.most[1][wave] = mv, sh.most[2][wave] = mq;
            }
            float mx = 0.0f;  // (a state whose products with the queries could pass float32)
            if (OUT && !F16) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(x[n][i]));
            }
            const bool any = __ballot(max(mk, mq) >= kHuge<T> || mv >= kHugeValue<T> || mx >= 0x1p64f) != 0;
            if (lane == 0) sh.odd[wave] = any;
        }
        __syncthreads();
        if (k + 1 < count) load(k + 1);
        if (wave == kWalkWaves - 1 && k + 1 < count) {
            put_decays<T>(sh.d[(k + 1) & 1], g, in, out, lane);
            if (k + 2 < count) load_decays(k + 2);
        }

        const float whole = d.whole;
        decay += d.all;
        int odd = d.odd;
#pragma unroll
        for (int i = 0; i < kWalkWaves; ++i) odd |= sh.odd[i];
        float most[3] = {0, 0, 0}, most_in = 0.0f, most_m = 0.0f;  // float16 only
        if constexpr (F16) {
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                uint32_t m = 0;
#pragma unroll
                for (int w = 0; w < kWalkWaves; ++w) m = max(m, sh.most[i][w]);
                most[i] = to_f(__builtin_bit_cast(f16, (uint16_t)m));
            }
            most_in = d.most_in * d.grow;
            most_m = most_in * d.most_out * most[0] * most[2] * (float)N;
            // M keeps 2^-50 of this, 2^-22 at least: beside a step of the lowest queries and keys ordinary ones
            // would lose theirs, and go row by row
            if (OUT) odd |= !(most_m < 0x1p28f);
        }
        auto from_state = [&](int h, f32x4 (&to)[HT]) {
#pragma unroll
            for (int t = 0; t < HT; ++t) to[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                Frag<T> f[HT];
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    const T* qp = sh.q + (16 * tile_of(h, t) + tl) * KS + 16 * (NT * half + n) + 4 * gl;
                    f[t] = NT > 1 ? pair_frag<T>(qp) : half_frag<T>(qp);
                }
                // (products that wait for each other's sums do not follow each other)
#pragma unroll
                for (int i = 0; i < K2; ++i)
#pragma unroll
                    for (int t = 0; t < HT; ++t) to[t] = mma<T>(state[n / 2][i], f[t], to[t]);
            }
        };
        float sm = 1.0f;
        if (OUT && !odd) {
            sm = to_range<T>(most_m);
            // what the state before the chunk gives: either half has the other one's results of half of the steps
            if (live) {
                f32x4 other[HT];
                from_state(1 - half, other);
#pragma unroll
                for (int t = 0; t < HT; ++t) sh.across[wave ^ 4][t][lane] = other[t];
            }
            // the pairs: tiles on the diagonal by the first waves, those below it by the others
            auto pairs = [&](int ti, int si) {
                f32x4 m = {0, 0, 0, 0};
                const T* kp = sh.k + (16 * si + tl) * KS + 8 * gl;
                const T* qp = sh.q + (16 * ti + tl) * KS + 8 * gl;
#pragma unroll
                for (int k0 = 0; k0 < KK; k0 += 2) {
                    Frag<T> kf[2], qf[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (k0 + i < KK) kf[i] = row_frag<T>(kp + 32 * (k0 + i)), qf[i] = row_frag<T>(qp + 32 * (k0 + i));
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (k0 + i < KK) m = mma<T>(kf[i], qf[i], m);
                }
                return m;
            };
            auto keep = [&](int ti, int si, const f32x4& m) {
                put_parts<T, K2>(sh.m + Pairs::row(ti >> 1, 16 * ti + tl) + 16 * si + 4 * gl, Pairs::kSize, m * sm);
            };
            if (wave < TT) {
                keep(wave, wave, pairs(wave, wave) * weights_within<T>(d, wave, lane));
            } else if (wave >= 4 && wave < kWalkWaves - 1) {  // (the last wave has the decays)
                for (int j = wave - 4; j < TT * (TT - 1) / 2; j += 3) {
                    const int ti = j < 1 ? 1 : j < 3 ? 2 : 3, si = j - ti * (ti - 1) / 2;
                    keep(ti, si, pairs(ti, si) * weights_across<T>(d, ti, si, lane));
                }
            }
            __syncthreads();
        }
        if (__builtin_expect(odd, 0)) {
            // An infinity or NaN among the inputs, or one that comes of their products, would reach
            // other rows through the products' zeros: the chunk goes row by row, as the formula says.
            // (A weight above one comes last, one below it first: then nothing passes float32 that the
            // formula keeps within it.  Seventeen times as long as by products: 4 x 2048 steps of 64 heads
            // 2.7 ms.)
            for (int r = REVERSE ? Q - nt : 0; r < (REVERSE ? Q : nt); ++r) {
                const float e = exp_f<kFine<T>>(d.g[r]), in_r = d.in[r], out_r = d.out[r];
                const bool in_first = fabsf(in_r) <= 1.0f, out_first = fabsf(out_r) <= 1.0f;
                const float in_a = in_first ? in_r : 1.0f, in_b = in_first ? 1.0f : in_r;
                const float out_a = out_first ? out_r : 1.0f, out_b = out_first ? 1.0f : out_r;
                const float v = to_f(sh.v[r * VS + 16 * pq + tl]);
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = 16 * (NT * half + n) + 4 * gl + i;
                        if (at < N && p0 + 16 * pq + tl < P) {  // (what does not exist stays zero)
                            x[n][i] = fmaf(x[n][i], e, in_a * to_f(sh.k[r * KS + at]) * v * in_b);
                            if (OUT) sum = fmaf(x[n][i], out_a * to_f(sh.q[r * KS + at]), sum);
                        }
                    }
                if (OUT) {
                    sum = across_rows(sum);
                    if (gl == 0) sh.sums[r & 1][half][16 * pq + tl] = sum;
                    __syncthreads();
                    if (half == 0 && gl == 0 && p0 + 16 * pq + tl < P) {
                        sum = (sum + sh.sums[r & 1][1][16 * pq + tl]) * out_b;
                        if (a.D) sum = fmaf(skip, v, sum);
                        const int o = REVERSE ? Q - 1 - r : r;
                        result[o * a.result.sl + tl * a.result.sn] = from_f<T>(sum);
                    }
                }
            }
        }
        if (live && !odd) {
            Frag<T> vf[SS];
#pragma unroll
            for (int s = 0; s < SS; ++s) vf[s] = column_frag<T>(sh.v + 32 * s * VS + 16 * pq, VS, lane);
            if (OUT) {
                struct __attribute__((aligned(4 * sizeof(T)))) Own { Quad<T> v; };
                const float um = reciprocal_of_power(sm), ux = reciprocal_of_power(sx);
                f32x4 within[HT], across[HT];
                from_state(half, across);
#pragma unroll
                for (int t = 0; t < HT; ++t) within[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = K2 - 1; i >= 0; --i) {
#pragma unroll
                    for (int s = SS - 1; s >= 0; --s)
#pragma unroll
                        for (int t = s; t < HT; ++t)
                            within[t] = mma<T>(vf[s], row_frag<T>(sh.m + Pairs::row(t, 16 * tile(t) + tl) + i * Pairs::kSize + 32 * s + 8 * gl), within[t]);
#pragma unroll
                    for (int t = 0; t < HT; ++t) within[t] *= i ? 1.0f / kLift<T> : 1.0f;
                }
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    const int r = 16 * tile(t) + tl, o = REVERSE ? Q - 1 - r : r;
                    across[t] += sh.across[wave][t][lane];
                    const float f = d.from[r] * ux;
                    f32x4 sum;
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = fmaf(across[t][i], f, within[t][i] * um);
                    if (a.D) {  // (in float32: on M's diagonal it would be rounded with M, alike in all steps)
                        const Own v4 = *reinterpret_cast<const Own*>(sh.v + r * VS + 16 * pq + 4 * gl);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] = fmaf(skip, to_f(get_of<T>(v4.v, i)), sum[i]);
                    }
                    const Quad<T> y = four_of<T>(sum);
                    const int there = P - (p0 + 16 * pq + 4 * gl);
                    if (vectors) {
                        if (o < nt && there > 0)
                            *reinterpret_cast<Quad<T>*>((char*)result + (uint32_t)o * ((uint32_t)a.result.sl * (uint32_t)sizeof(T)) +
                                                     4u * gl * (uint32_t)sizeof(T)) = y;
                    } else {
                        T* to = result + o * a.result.sl + 4 * gl * a.result.sn;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (o < nt && i < there) to[i * a.result.sn] = get_of<T>(y, i);
                    }
                }
            }
            // the state after the chunk
            const float sv = to_range<T>(most_in * most[1]), uv = reciprocal_of_power(sv);
            Frag<T> part[SS][kParts<T>];
#pragma unroll
            for (int s = 0; s < SS; ++s) {
                const f32x4* to = reinterpret_cast<const f32x4*>(&d.to[32 * s + 8 * gl]);
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = frag_get<T>(vf[s], j) * (to[j / 4][j % 4] * sv);
                split<T>(w, part[s]);
            }
            // (the tiles in turn: products that wait for each other's sums do not follow each other)
            f32x4 add[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) add[n] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < SS; ++s) {
                Frag<T> kf[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) kf[n] = column_frag<T>(sh.k + 32 * s * KS + 16 * (NT * half + n), KS, lane);
#pragma unroll
                for (int i = 0; i < kParts<T>; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) add[n] = mma<T>(kf[n], part[s][i], add[n]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = fmaf(x[n][i], whole, add[n][i] * uv);
        }
        if (F16 && OUT) most_state();
        if (OUT) result += (REVERSE ? -Q : Q) * a.result.sl;
    }
    if (ENDS) {
        put(a.seg_x, item, 1.0f);
        if (pb == 0 && threadIdx.x == 0) a.seg_decay[item * a.H + h] = (float)decay;
    } else if (a.x_out && pos == segments - 1) {
        // backwards: the gradient of the state before the first step
        put(a.x_out, it.state, REVERSE && len > 0 ? exp_f<kFine<T>>(gs[it.beg * a.g.sl]) : 1.0f);
    }
}

template <class T, int NP, bool REVERSE, bool FAST>
static void launch_walk_lay(const WalkArgs& a, hipStream_t s) {
    const int64_t blocks = (a.P + kWalkValues - 1) / kWalkValues;
    const dim3 grid((unsigned)(a.items * a.H * blocks)), wg(kWalkThreads);
    if (a.segment < a.q.L) hipLaunchKernelGGL((linear_walk_kernel<T, NP, false, REVERSE, true, FAST>), grid, wg, 0, s, a);
    if (a.result.data) hipLaunchKernelGGL((linear_walk_kernel<T, NP, true, REVERSE, false, FAST>), grid, wg, 0, s, a);
    else if (!REVERSE) hipLaunchKernelGGL((linear_walk_kernel<T, NP, false, false, false, FAST>), grid, wg, 0, s, a);
}
template <class T, int NP, bool REVERSE>
static hipError_t launch_walk_keys(const WalkArgs& a, hipStream_t s) {
    if (a.fast) launch_walk_lay<T, NP, REVERSE, true>(a, s);
    else launch_walk_lay<T, NP, REVERSE, false>(a, s);
    return hipGetLastError();
}
template <class T, bool REVERSE>
hipError_t launch_walk(const WalkArgs& a, hipStream_t s) {
    if (a.N <= 32) return launch_walk_keys<T, 32, REVERSE>(a, s);
    if (a.N <= 64) return launch_walk_keys<T, 64, REVERSE>(a, s);
    if (a.N <= 128) return launch_walk_keys<T, 128, REVERSE>(a, s);
    return launch_walk_keys<T, 256, REVERSE>(a, s);
}

}  // namespace ssm

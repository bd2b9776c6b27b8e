// The walk over the chunks of a sequence, for linear attention forwards and for the
// gradient of its values backwards (include/ssm.h: ssm_linear_attention).
#pragma once

#include "linear.hpp"

namespace ssm {

constexpr int kWalkThreads = 256;
constexpr int kWalkValues = 64;  // values of a workgroup: 16 to a wave

// A workgroup has one head, 64 of its values and one segment of a sequence, and takes a
// chunk of rows at a time.  With the pairs' weights M_ts = out_t (q_t . k_s) E_ts in_s
// (s <= t, D on the diagonal) the chunk's results are
//   result_t = sum_s M_ts value_s + out_t E_t x^T q_t,
// and the state becomes E x + sum_s E'_s in_s k_s value_s^T: four matrix products.  A wave
// has the whole state of its 16 values in float32 in registers, in the order in which the
// matrix instruction leaves it and in which, rounded, it is the next chunk's operand: the
// state goes through no memory.  M goes through LDS once, a tile of rows from each wave.
// Rounding to the activations' type: M and the state as operands for the results, which
// are rounded to it anyway.  What is added to the state is split into two parts of that
// type, so that the state has 16 (bf16) or 22 (f16) bits of every product.
// ENDS: the first of two passes, which finds each segment's end state for the second.
// OUT: results wanted.
template <class T, int NP, bool OUT, bool REVERSE, bool ENDS>
__global__ __launch_bounds__(kWalkThreads) void linear_walk_kernel(const WalkArgs a) {
    constexpr int Q = kChunk<T>, TT = Q / 16, KK = NP / 32, SS = Q / 32, NT = NP / 16;
    constexpr int KS = NP + kRoom<T>, VS = kWalkValues + kRoom<T>, MS = Q + kRoom<T>;
    struct __attribute__((aligned(16))) Shared {
        T k[Q * KS];
        T v[Q * VS];
        T q[OUT ? Q * KS : 8];
        T m[OUT ? Q * MS : 8];
        Decays<T> d;
        uint32_t most[3][4];
        int odd[4];
    };
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tl = lane & 15, gl = lane >> 4;
    const int blocks = (int)((a.P + kWalkValues - 1) / kWalkValues);
    const int64_t bid = blockIdx.x;
    const int pb = (int)(bid % blocks), h = (int)(bid / blocks % a.H);
    const int64_t item = bid / blocks / a.H;
    Item it;
    if (!find_item(a.q, item, (int)a.segment, it) || it.state < 0) return;
    const int len = it.end - it.beg, segments = chunks_of(len, (int)a.segment);
    if (it.c >= segments) return;
    const int pos = REVERSE ? segments - 1 - it.c : it.c;  // in the order of the walk
    const int chunks = (len + Q - 1) / Q, per = (int)(a.segment / Q);
    const int c0 = it.c * per, c1 = min(c0 + per, chunks);

    const int N = (int)a.N, P = (int)a.P;
    const int p0 = pb * kWalkValues, p = p0 + 16 * wave + tl;
    const bool live = p0 + 16 * wave < P;
    f32x4 x[NT];
    // the lane's states of a row of a [rows, H, N, P] array: n = 16 tile + 4 gl + i, value p
    auto place = [&](int64_t r) { return ((r * a.H + h) * N + 4 * gl) * P + p; };
    auto get = [&](const float* from) {
        const float* f = from + (p < P ? 0 : P - 1 - p);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[n][i] = 16 * n + 4 * gl + i < N && p < P ? f[(int64_t)(16 * n + i) * P] : 0.0f;
    };
    auto put = [&](float* to, float factor) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * n + 4 * gl + i < N && p < P) to[(int64_t)(16 * n + i) * P] = x[n][i] * factor;
    };
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] = f32x4{0, 0, 0, 0};
    };
    // the item of the segment at a place of the walk
    auto item_at = [&](int j) { return item - it.c + (REVERSE ? segments - 1 - j : j); };
    float decay = 1.0f;  // of the segment
    if (ENDS) {
        if (segments == 1) return;
        if (pos == 0 || pos == segments - 1) {
            // the last one's end is not needed: its place keeps the initial state, which the
            // final state may overwrite while the second pass still needs it
            if (a.x_in) get(a.x_in + place(it.state));
            else clear();
            if (pos != 0) {
                put(a.seg_x + place(item), 1.0f);
                return;
            }
        } else {
            clear();
        }
    } else if (segments == 1) {
        if (a.x_in) get(a.x_in + place(it.state));
        else clear();
    } else {
        get(a.seg_x + place(item_at(pos == 0 ? segments - 1 : 0)));
        for (int j = 1; j < pos; ++j) {
            const int64_t before = item_at(j);
            const float e = a.seg_decay[before * a.H + h];
            f32x4 y[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) y[n] = x[n];
            get(a.seg_x + place(before));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = fmaf(y[n][i], e, x[n][i]);
        }
    }

    const int grp = (int)(h / (a.H / a.G));
    const T* key = (const T*)a.key.data + it.row * a.key.sb + grp * a.key.sg;
    const T* query = (const T*)a.query.data + it.row * a.query.sb + grp * a.query.sg;
    const T* value = (const T*)a.value.data + it.row * a.value.sb + h * a.value.sg + p0 * a.value.sn;
    T* result = (T*)a.result.data + it.row * a.result.sb + h * a.result.sg;
    const float* gs = (const float*)a.g.data + it.row * a.g.sb + h * a.g.sh;
    const float* bs = a.beta.data ? (const float*)a.beta.data + it.row * a.beta.sb + h * a.beta.sh : nullptr;
    const float skip = a.D ? a.D[h] : 0.0f;
    const int64_t Pp = (a.P + 31) / 32 * 32;
    float* saved = a.saved && !ENDS ? a.saved + ((linear_row(a.q, it, Q) * a.H + h) * N + 4 * gl) * Pp + p : nullptr;

    Carrier<T, NP, kWalkThreads> ck, cq;
    Carrier<T, kWalkValues, kWalkThreads> cv;
    float g = 0.0f, in = 0.0f, out = 0.0f;
    auto load = [&](int c) {
        const int t0 = it.beg + c * Q, nt = min(Q, it.end - t0);
        ck.load(key + t0 * a.key.sl, a.key_lay, a.key.sn, a.key.sl, N, nt, tid);
        cv.load(value + t0 * a.value.sl, a.value_lay, a.value.sn, a.value.sl, P - p0, nt, tid);
        if (OUT) cq.load(query + t0 * a.query.sl, a.query_lay, a.query.sn, a.query.sl, N, nt, tid);
        if (wave == 0) {
            const int o = REVERSE ? Q - 1 - lane : lane, t = t0 + o;
            g = in = out = 0.0f;
            if (lane < Q && o < nt) {
                const float b = bs ? bs[t * a.beta.sl] : 1.0f;
                const int tg = REVERSE ? t + 1 : t;
                g = tg < it.end ? gs[tg * a.g.sl] : 0.0f;
                in = REVERSE ? a.scale : b;
                out = REVERSE ? b : a.scale;
            }
        }
    };

    const int count = c1 - c0;
    if (count > 0) load(REVERSE ? c1 - 1 : c0);
    for (int k = 0; k < count; ++k) {
        const int c = REVERSE ? c1 - 1 - k : c0 + k;
        const int t0 = it.beg + c * Q, nt = min(Q, it.end - t0);
        if (saved && p < Pp) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (16 * n + 4 * gl + i < N)
                        saved[(int64_t)c * a.H * N * Pp + (16 * n + i) * Pp] = p < P ? x[n][i] : 0.0f;
        }
        __syncthreads();  // the last chunk's tiles have been read
        ck.template store<REVERSE>(sh.k, a.key_lay, tid);
        cv.template store<REVERSE>(sh.v, a.value_lay, tid);
        if (OUT) cq.template store<REVERSE>(sh.q, a.query_lay, tid);
        if (wave == 0) put_decays<T>(sh.d, g, in, out, lane);
        {
            uint32_t mk = ck.most(), mv = cv.most(), mq = OUT ? cq.most() : 0;
            if constexpr (std::is_same<T, f16>::value) {
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    mk = max(mk, (uint32_t)__shfl_xor((int)mk, d)), mv = max(mv, (uint32_t)__shfl_xor((int)mv, d));
                    if (OUT) mq = max(mq, (uint32_t)__shfl_xor((int)mq, d));
                }
                if (lane == 0) sh.most[0][wave] = mk, sh.most[1][wave] = mv, sh.most[2][wave] = mq;
            }
            const bool any = __ballot(max(max(mk, mv), mq) >= kInf<T>) != 0;
            if (lane == 0) sh.odd[wave] = any;
        }
        __syncthreads();
        if (k + 1 < count) load(REVERSE ? c - 1 : c + 1);

        const float whole = sh.d.whole;
        decay *= whole;
        if (sh.d.odd | sh.odd[0] | sh.odd[1] | sh.odd[2] | sh.odd[3]) {
            // An infinity or NaN among the inputs would reach earlier rows through the products'
            // zeros: the chunk goes row by row, as the formula says.
            for (int r = REVERSE ? Q - nt : 0; r < (REVERSE ? Q : nt); ++r) {
                const float e = exp_f<kFine<T>>(sh.d.g[r]), in_r = sh.d.in[r];
                const float v = to_f(sh.v[r * VS + 16 * wave + tl]);
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = 16 * n + 4 * gl + i;
                        if (at < N) {
                            x[n][i] = fmaf(x[n][i], e, in_r * to_f(sh.k[r * KS + at]) * v);
                            if (OUT) sum = fmaf(x[n][i], to_f(sh.q[r * KS + at]), sum);
                        }
                    }
                if (OUT) {
                    sum = across_rows(sum) * sh.d.out[r];
                    if (a.D) sum = fmaf(skip, v, sum);
                    const int t = t0 + (REVERSE ? Q - 1 - r : r);
                    if (gl == 0 && p < P) result[t * a.result.sl + p * a.result.sn] = from_f<T>(sum);
                }
            }
            continue;
        }

        float most[3] = {0, 0, 0};
        if constexpr (std::is_same<T, f16>::value) {
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint32_t m = max(max(sh.most[i][0], sh.most[i][1]), max(sh.most[i][2], sh.most[i][3]));
                most[i] = to_f(__builtin_bit_cast(f16, (uint16_t)m));
            }
        }
        const float most_in = sh.d.most_in * sh.d.grow, most_out = sh.d.most_out;  // float16 only
        f32x4 across[OUT ? TT : 1];
        float sm = 1.0f, sx = 1.0f;
        if (OUT) {
            sm = to_range<T>(most_in * most_out * most[0] * most[2] * (float)N + fabsf(skip));
            // what the state before the chunk gives
            if (live) {
                if constexpr (std::is_same<T, f16>::value) {
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
                    sx = to_range<T>(m);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) across[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = x[2 * kk][i] * sx, e[4 + i] = x[2 * kk + 1][i] * sx;
                    const Frag<T> f = frag_of<T>(e);
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        across[t] = mma<T>(f, pair_frag<T>(sh.q + (16 * t + tl) * KS + 32 * kk + 4 * gl), across[t]);
                }
            }
            // the pairs' weights: a wave has rows 16 ti .. + 15, or half of them
            const int ti = wave % TT;
            Frag<T> qf[KK];
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) qf[kk] = row_frag<T>(sh.q + (16 * ti + tl) * KS + 32 * kk + 8 * gl);
#pragma unroll
            for (int j = 0; j < TT * TT / 4; ++j) {
                const int si = wave / TT + j * (4 / TT);
                f32x4 m = {0, 0, 0, 0};
                if (si <= ti) {
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
                        m = mma<T>(row_frag<T>(sh.k + (16 * si + tl) * KS + 32 * kk + 8 * gl), qf[kk], m);
                    m *= pair_weights<T>(sh.d, ti, si, lane);
                    if (si == ti) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) m[i] += 4 * gl + i == tl ? skip : 0.0f;
                    }
                }
                struct __attribute__((aligned(4 * sizeof(T)))) Four { T v[4]; } w;
#pragma unroll
                for (int i = 0; i < 4; ++i) w.v[i] = from_f<T>(m[i] * sm);
                *reinterpret_cast<Four*>(sh.m + (16 * ti + tl) * MS + 16 * si + 4 * gl) = w;
            }
            __syncthreads();
        }
        if (!live) continue;
        Frag<T> vf[SS];
#pragma unroll
        for (int s = 0; s < SS; ++s) vf[s] = column_frag<T>(sh.v + 32 * s * VS + 16 * wave, VS, lane);
        if (OUT) {
            const float um = reciprocal_of_power(sm), ux = reciprocal_of_power(sx);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                f32x4 within = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s <= t / 2; ++s)
                    within = mma<T>(vf[s], row_frag<T>(sh.m + (16 * t + tl) * MS + 32 * s + 8 * gl), within);
                const int r = 16 * t + tl, o = REVERSE ? Q - 1 - r : r;
                const float f = sh.d.from[r] * ux;
                if (o < nt) {
                    T* to = result + (t0 + o) * a.result.sl + (p0 + 16 * wave + 4 * gl) * a.result.sn;
                    const int there = P - (p0 + 16 * wave + 4 * gl);
                    Vec4<T> y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y.v[i] = from_f<T>(fmaf(across[t][i], f, within[i] * um));
                    if (there >= 4 && a.result.sn == 1) {
                        *reinterpret_cast<Vec4<T>*>(to) = y;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < there) to[i * a.result.sn] = y.v[i];
                    }
                }
            }
        }
        // the state after the chunk
        const float sv = to_range<T>(most_in * most[1]), uv = reciprocal_of_power(sv);
        Frag<T> hi[SS], lo[SS];
#pragma unroll
        for (int s = 0; s < SS; ++s) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = frag_get<T>(vf[s], j) * (sh.d.to[32 * s + 8 * gl + j] * sv);
            split<T>(w, hi[s], lo[s]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 add = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < SS; ++s) {
                const Frag<T> kf = column_frag<T>(sh.k + 32 * s * KS + 16 * n, KS, lane);
                add = mma<T>(kf, hi[s], add);
                if (kSplit<T>) add = mma<T>(kf, lo[s], add);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = fmaf(x[n][i], whole, add[i] * uv);
        }
    }
    if (ENDS) {
        put(a.seg_x + place(item), 1.0f);
        if (pb == 0 && tid == 0) a.seg_decay[item * a.H + h] = decay;
    } else if (a.x_out && pos == segments - 1) {
        // backwards: the gradient of the state before the first step
        const float e = REVERSE && len > 0 ? exp_f<kFine<T>>(gs[it.beg * a.g.sl]) : 1.0f;
        put(a.x_out + place(it.state), e);
    }
}

template <class T, int NP, bool REVERSE>
hipError_t launch_walk_keys(const WalkArgs& a, hipStream_t s) {
    const int64_t blocks = (a.P + kWalkValues - 1) / kWalkValues;
    const dim3 grid((unsigned)(a.items * a.H * blocks)), wg(kWalkThreads);
    if (a.segment < a.q.L) hipLaunchKernelGGL((linear_walk_kernel<T, NP, false, REVERSE, true>), grid, wg, 0, s, a);
    if (a.result.data) hipLaunchKernelGGL((linear_walk_kernel<T, NP, true, REVERSE, false>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((linear_walk_kernel<T, NP, false, REVERSE, false>), grid, wg, 0, s, a);
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

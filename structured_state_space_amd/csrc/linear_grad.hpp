// The gradients of linear attention's queries, keys, decays and weights
// (include/ssm.h: ssm_linear_attention_backward), from the states before every chunk and
// the gradients of the states behind them.
#pragma once

#include "linear.hpp"

namespace ssm {

constexpr int kPairValues = 64;
template <int NP>
constexpr int kPairThreads = NP > 128 ? 512 : 256;

// A workgroup has one chunk of a sequence and some of a group's heads, whose gradients of
// the shared queries and keys it adds up in registers.  Per head, with E_ts as in the walk,
// u_ts = scale E_ts, x the state before the chunk and X the gradient of the one behind it:
//   dM_ts = dy_t . v_s,   W_ts = u_ts (q_t . k_s) dM_ts              (s <= t)
//   dq_t = sum_s u_ts beta_s dM_ts k_s + scale E_t x dy_t            = within + before_t
//   dk_s = beta_s (sum_t u_ts dM_ts q_t + E'_s X v_s)                = beta_s (within + behind_s)
//   dbeta_s = sum_t W_ts + k_s . behind_s
//   dg_r = sum over pairs t >= r > s of beta_s W_ts, over t >= r of q_t . before_t, over s < r of
//          beta_s k_s . behind_s, and E <x, X>:
// a step's decay takes part in every product over it.  All of dg and dbeta are sums in
// float32 of float32 numbers: x and X are split into two operands of the activations' type,
// and only u beta dM is rounded to it, for dq and dk, which are of that type.
// Values beyond 64 go block by block; every sum is linear in them.  q_t . k_s is formed
// once for all heads.  Results lie transposed (lane: step, registers: four keys), so that
// rows of four keys are multiplied with q and k and stored at once.
template <class T, int NP>
__global__ __launch_bounds__(kPairThreads<NP>) void linear_pairs_kernel(const PairArgs a) {
    constexpr int TH = kPairThreads<NP>, W = TH / 64;
    constexpr int Q = kChunk<T>, TT = Q / 16, KK = NP / 32, SS = Q / 32, PK = kPairValues / 32;
    constexpr int NT = NP / 16 < W ? 1 : NP / 16 / W;             // tiles of keys of a wave
    constexpr int OWN = TT * TT < W ? 1 : TT * TT / W, STEP = W / TT;  // tiles of pairs of a wave
    constexpr int KS = NP + kRoom<T>, VS = kPairValues + kRoom<T>, MS = Q + kRoom<T>;
    struct __attribute__((aligned(16))) Shared {
        T q[Q * KS], k[Q * KS], v[Q * VS], dy[Q * VS], m[Q * MS];
        Decays<T> d;
        float beta[Q];
        float rows[STEP][Q], columns[TT][Q], diagonal[Q], skip[TT];  // sums of W over its rows and columns
        float before[W][Q], behind[W][Q], whole[W];
        float next, most_beta;  // the decay from the chunk's last step to the next one
        uint32_t most[2][W];
    };
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tl = lane & 15, gl = lane >> 4;
    const int64_t bid = blockIdx.x;
    const int blk = (int)(bid % a.blocks), grp = (int)(bid / a.blocks % a.G);
    const int64_t item = bid / a.blocks / a.G;
    const int Hg = (int)(a.H / a.G), h0 = grp * Hg + blk * a.heads, h1 = min(h0 + a.heads, (grp + 1) * Hg);
    Item it;
    const bool found = find_item(a.q, item, Q, it);
    const int t0 = found ? it.beg + it.c * Q : 0, nt = found ? min(Q, it.end - t0) : 0;
    if (nt <= 0) {
        if (a.skips && h0 + tid < h1)
            for (int h = h0 + tid; h < h1; h += TH) a.skips[item * a.H + h] = 0.0f;
        return;
    }
    const int N = (int)a.N, P = (int)a.P, values = (P + kPairValues - 1) / kPairValues;
    const int64_t Pp = (a.P + 31) / 32 * 32, row = linear_row(a.q, it, Q) + it.c;

    {
        Carrier<T, NP, TH> c;
        c.load((const T*)a.qv.data + it.row * a.qv.sb + grp * a.qv.sg + t0 * a.qv.sl, a.q_lay, a.qv.sn, a.qv.sl, N, nt, tid);
        c.template store<false>(sh.q, a.q_lay, tid);
        c.load((const T*)a.k.data + it.row * a.k.sb + grp * a.k.sg + t0 * a.k.sl, a.k_lay, a.k.sn, a.k.sl, N, nt, tid);
        c.template store<false>(sh.k, a.k_lay, tid);
    }
    Carrier<T, kPairValues, TH> cv, cy;
    float g = 0.0f, beta = 0.0f, g_next = 0.0f;
    auto load = [&](int h, int pb) {
        const int p0 = pb * kPairValues;
        cv.load((const T*)a.v.data + it.row * a.v.sb + h * a.v.sg + t0 * a.v.sl + p0 * a.v.sn, a.v_lay, a.v.sn, a.v.sl, P - p0,
                nt, tid);
        cy.load((const T*)a.dy.data + it.row * a.dy.sb + h * a.dy.sg + t0 * a.dy.sl + p0 * a.dy.sn, a.dy_lay, a.dy.sn, a.dy.sl,
                P - p0, nt, tid);
        if (wave == 0) {
            const float* gs = (const float*)a.g.data + it.row * a.g.sb + h * a.g.sh;
            g = beta = 0.0f;
            if (lane < nt) {
                g = gs[(t0 + lane) * a.g.sl];
                beta = a.beta.data ? ((const float*)a.beta.data)[it.row * a.beta.sb + h * a.beta.sh + (t0 + lane) * a.beta.sl] : 1.0f;
            }
            // what lies between the chunk and the state behind the next step
            g_next = t0 + nt < it.end ? gs[(t0 + nt) * a.g.sl] : 0.0f;
        }
    };
    load(h0, 0);
    __syncthreads();

    const int ti = wave % TT, si0 = wave / TT;
    f32x4 qk[OWN];
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int si = si0 + j * STEP;
        qk[j] = f32x4{0, 0, 0, 0};
        if (si <= ti) {
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                qk[j] = mma<T>(row_frag<T>(sh.k + (16 * si + tl) * KS + 32 * kk + 8 * gl),
                               row_frag<T>(sh.q + (16 * ti + tl) * KS + 32 * kk + 8 * gl), qk[j]);
        }
    }
    f32x4 dq[NT][TT], dk[NT][TT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TT; ++t) dq[n][t] = dk[n][t] = f32x4{0, 0, 0, 0};
    const int n0 = 16 * NT * wave;  // the wave's first key

    // wave 0, lane r: sums over the blocks of a head's values
    float sum_row = 0.0f, sum_column = 0.0f, sum_diagonal = 0.0f, sum_before = 0.0f, sum_behind = 0.0f, sum_whole = 0.0f,
          sum_skip = 0.0f;
    float g_own = 0.0f, beta_own = 0.0f, across = 1.0f;
    auto collect = [&]() {
        if (lane < Q) {
#pragma unroll
            for (int i = 0; i < STEP; ++i) sum_row += sh.rows[i][lane];
#pragma unroll
            for (int i = 0; i < TT; ++i) sum_column += sh.columns[i][lane];
            sum_diagonal += sh.diagonal[lane];
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (16 * NT * i < NP) sum_before += sh.before[i][lane], sum_behind += sh.behind[i][lane];
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (16 * NT * i < NP) sum_whole += sh.whole[i];
#pragma unroll
        for (int i = 0; i < TT; ++i) sum_skip += sh.skip[i];
    };
    auto finish = [&](int h) {
        // sums over the steps from r on, and before r
        float from = sum_row + sum_before - beta_own * sum_column, till = beta_own * sum_behind;
        const float own = till;
#pragma unroll
        for (int d = 1; d < Q; d <<= 1) {
            const float f = __shfl_down(from, d), b = __shfl_up(till, d);
            if (lane + d < Q) from += f;
            if (lane >= d) till += b;
        }
        const float dg = from + (till - own) + across * sum_whole;
        if (lane < nt) {
            // a reset takes part in no product, and the sums' rounding is not left in its place
            ((float*)a.dg.data)[it.row * a.dg.sb + h * a.dg.sh + (t0 + lane) * a.dg.sl] =
                exp_f<kFine<T>>(g_own) == 0.0f ? 0.0f : dg;
            if (a.dbeta.data)
                ((float*)a.dbeta.data)[it.row * a.dbeta.sb + h * a.dbeta.sh + (t0 + lane) * a.dbeta.sl] =
                    sum_column + sum_diagonal + sum_behind;
        }
        if (a.skips && lane == 0) a.skips[item * a.H + h] = sum_skip;
        sum_row = sum_column = sum_diagonal = sum_before = sum_behind = sum_whole = sum_skip = 0.0f;
    };

    const int count = (h1 - h0) * values;
    int h = h0, pb = 0;
    for (int k = 0; k < count; ++k) {
        // the states' fragments: keys n0 + 16 n + tl, values 32 kk + 8 gl .. + 7
        float x[NT][PK][8], X[NT][PK][8];
        const int p0 = pb * kPairValues;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int kk = 0; kk < PK; ++kk) {
                const int key = n0 + 16 * n + tl, p = p0 + 32 * kk + 8 * gl;
                f32x4 v[4] = {};
                if (key < N && p < Pp) {
                    const int64_t at = ((row * a.H + h) * N + key) * Pp + p;
                    const f32x4* s = reinterpret_cast<const f32x4*>(a.states + at);
                    const f32x4* e = reinterpret_cast<const f32x4*>(a.ahead + at);
                    v[0] = s[0], v[1] = s[1], v[2] = e[0], v[3] = e[1];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[n][kk][i] = v[0][i], x[n][kk][4 + i] = v[1][i], X[n][kk][i] = v[2][i], X[n][kk][4 + i] = v[3][i];
            }
        if (k) __syncthreads();  // the last block's tiles have been read, its sums are there
        cv.template store<false>(sh.v, a.v_lay, tid);
        cy.template store<false>(sh.dy, a.dy_lay, tid);
        if constexpr (std::is_same<T, f16>::value) {
            uint32_t mv = cv.most(), my = cy.most();
#pragma unroll
            for (int d = 1; d < 64; d <<= 1)
                mv = max(mv, (uint32_t)__shfl_xor((int)mv, d)), my = max(my, (uint32_t)__shfl_xor((int)my, d));
            if (lane == 0) sh.most[0][wave] = mv, sh.most[1][wave] = my;
        }
        if (wave == 0) {
            if (k) {
                collect();
                if (pb == 0) finish(h - 1);
            }
            if (pb == 0) {
                put_decays<T>(sh.d, g, lane < nt ? 1.0f : 0.0f, lane < nt ? a.scale : 0.0f, lane);
                if (lane < Q) sh.beta[lane] = beta;
                g_own = g, beta_own = beta;
                across = exp_f<kFine<T>>(across_rows(row_sum(g)) + g_next);
                if (lane == 0) sh.next = exp_f<kFine<T>>(g_next);
                if constexpr (std::is_same<T, f16>::value) {
                    float m = fabsf(beta);
#pragma unroll
                    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
                    if (lane == 0) sh.most_beta = m;
                }
            }
        }
        __syncthreads();
        if (++pb == values) pb = 0, ++h;
        if (k + 1 < count) load(h, pb);

        float sm = 1.0f;
        if constexpr (std::is_same<T, f16>::value) {
            uint32_t mv = 0, my = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) mv = max(mv, sh.most[0][i]), my = max(my, sh.most[1][i]);
            sm = to_range<T>(fabsf(a.scale) * sh.d.grow * sh.most_beta * (float)kPairValues *
                             to_f(__builtin_bit_cast(f16, (uint16_t)mv)) * to_f(__builtin_bit_cast(f16, (uint16_t)my)));
        }
        // the pairs
        float row_part = 0.0f, skip = 0.0f;
        {
            Frag<T> yf[PK];
#pragma unroll
            for (int kk = 0; kk < PK; ++kk) yf[kk] = row_frag<T>(sh.dy + (16 * ti + tl) * VS + 32 * kk + 8 * gl);
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const int si = si0 + j * STEP;
                if (si >= TT) break;
                struct __attribute__((aligned(4 * sizeof(T)))) Four { T v[4]; } w;
                float column[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) w.v[i] = from_f<T>(0.0f);
                if (si <= ti) {
                    f32x4 dm = {0, 0, 0, 0};
#pragma unroll
                    for (int kk = 0; kk < PK; ++kk)
                        dm = mma<T>(row_frag<T>(sh.v + (16 * si + tl) * VS + 32 * kk + 8 * gl), yf[kk], dm);
                    const f32x4 u = pair_weights<T>(sh.d, ti, si, lane);
                    const f32x4 b = *reinterpret_cast<const f32x4*>(&sh.beta[16 * si + 4 * gl]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float um = u[i] * dm[i], wt = um * qk[j][i];
                        const bool diagonal = si == ti && 4 * gl + i == tl;
                        if (diagonal) {
                            sh.diagonal[16 * ti + tl] = wt;
                            skip = dm[i];
                        } else {
                            row_part = fmaf(wt, b[i], row_part);
                            column[i] = wt;
                        }
                        w.v[i] = from_f<T>(um * b[i] * sm);
                    }
                }
                *reinterpret_cast<Four*>(sh.m + (16 * ti + tl) * MS + 16 * si + 4 * gl) = w;
#pragma unroll
                for (int i = 0; i < 4; ++i) column[i] = row_sum(column[i]);
                if (tl == 0) *reinterpret_cast<f32x4*>(&sh.columns[ti][16 * si + 4 * gl]) = f32x4{column[0], column[1], column[2], column[3]};
            }
            row_part = across_rows(row_part);
            skip = across_rows(row_sum(skip));
            if (gl == 0) sh.rows[si0][16 * ti + tl] = row_part;
            if (lane == 0 && si0 <= ti && (ti - si0) % STEP == 0) sh.skip[ti] = skip;  // it has the diagonal's tile
        }
        __syncthreads();
        if (n0 >= NP) continue;

        // keys by steps: dq and dk
        float before[TT], behind[TT], whole = 0.0f;
#pragma unroll
        for (int t = 0; t < TT; ++t) before[t] = behind[t] = 0.0f;
        const float um = reciprocal_of_power(sm);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int key = n0 + 16 * n;
            Frag<T> kf[SS], qf[SS], xh[PK], xl[PK], Xh[PK], Xl[PK];
#pragma unroll
            for (int s = 0; s < SS; ++s) {
                kf[s] = column_frag<T>(sh.k + 32 * s * KS + key, KS, lane);
                qf[s] = column_frag<T>(sh.q + 32 * s * KS + key, KS, lane);
            }
            float sx = 1.0f, sX = 1.0f;
            if constexpr (std::is_same<T, f16>::value) {
                float mx = 0.0f, mX = 0.0f;
#pragma unroll
                for (int kk = 0; kk < PK; ++kk)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float u = fabsf(x[n][kk][i]), v = fabsf(X[n][kk][i]);
                        mx = fmaxf(mx, u < INFINITY ? u : 0.0f), mX = fmaxf(mX, v < INFINITY ? v : 0.0f);
                    }
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d)), mX = fmaxf(mX, __shfl_xor(mX, d));
                sx = to_range<T>(mx), sX = to_range<T>(mX);
            }
#pragma unroll
            for (int kk = 0; kk < PK; ++kk) {
                float u[8], v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    whole = fmaf(x[n][kk][i], X[n][kk][i], whole);
                    u[i] = x[n][kk][i] * sx, v[i] = X[n][kk][i] * sX;
                }
                split<T>(u, xh[kk], xl[kk]);
                split<T>(v, Xh[kk], Xl[kk]);
            }
            const float ux = reciprocal_of_power(sx), uX = reciprocal_of_power(sX);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                f32x4 in = {0, 0, 0, 0}, out = {0, 0, 0, 0};
#pragma unroll
                for (int kk = 0; kk < PK; ++kk) {
                    const Frag<T> yf = row_frag<T>(sh.dy + (16 * t + tl) * VS + 32 * kk + 8 * gl);
                    const Frag<T> vf = row_frag<T>(sh.v + (16 * t + tl) * VS + 32 * kk + 8 * gl);
                    in = mma<T>(xh[kk], yf, in), out = mma<T>(Xh[kk], vf, out);
                    if (kSplit<T>) in = mma<T>(xl[kk], yf, in), out = mma<T>(Xl[kk], vf, out);
                }
                f32x4 wq = {0, 0, 0, 0}, wk = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < SS; ++s) {
                    if (s <= t / 2) wq = mma<T>(kf[s], row_frag<T>(sh.m + (16 * t + tl) * MS + 32 * s + 8 * gl), wq);
                    if (s >= t / 2) wk = mma<T>(qf[s], column_frag<T>(sh.m + 32 * s * MS + 16 * t, MS, lane), wk);
                }
                const int r = 16 * t + tl;
                const float from = sh.d.from[r] * ux, to = sh.d.to[r] * sh.next * uX, b = sh.beta[r];
                struct __attribute__((aligned(4 * sizeof(T)))) Four { T v[4]; };
                const Four q4 = *reinterpret_cast<const Four*>(sh.q + r * KS + key + 4 * gl);
                const Four k4 = *reinterpret_cast<const Four*>(sh.k + r * KS + key + 4 * gl);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = in[i] * from, v = out[i] * to;
                    before[t] = fmaf(u, to_f(q4.v[i]), before[t]);
                    behind[t] = fmaf(v, to_f(k4.v[i]), behind[t]);
                    dq[n][t][i] += fmaf(wq[i], um, u);
                    dk[n][t][i] += fmaf(wk[i], um, v * b);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            before[t] = across_rows(before[t]), behind[t] = across_rows(behind[t]);
            if (gl == 0) sh.before[wave][16 * t + tl] = before[t], sh.behind[wave][16 * t + tl] = behind[t];
        }
        whole = across_rows(row_sum(whole));
        if (lane == 0) sh.whole[wave] = whole;
    }
    __syncthreads();
    if (wave == 0) {
        collect();
        finish(h1 - 1);
    }
    if (n0 >= NP) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int r = 16 * t + tl, key = n0 + 16 * n + 4 * gl, there = N - key;
            if (r >= nt || there <= 0) continue;
            if (a.blocks > 1) {
                const int64_t all = a.Bsz * a.G * a.q.L * N;
                float* to = a.parts + blk * 2 * all + (((int64_t)it.row * a.G + grp) * a.q.L + t0 + r) * N + key;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < there) to[i] = dq[n][t][i], to[all + i] = dk[n][t][i];
            } else {
                T* q = (T*)a.dq.data + it.row * a.dq.sb + grp * a.dq.sg + (t0 + r) * a.dq.sl + key * a.dq.sn;
                T* k = (T*)a.dk.data + it.row * a.dk.sb + grp * a.dk.sg + (t0 + r) * a.dk.sl + key * a.dk.sn;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < there) q[i * a.dq.sn] = from_f<T>(dq[n][t][i]), k[i * a.dk.sn] = from_f<T>(dk[n][t][i]);
            }
        }
}

// The sums over a group's workgroups, and of D's gradient over the chunks (in float64).
template <class T>
__global__ __launch_bounds__(256) void linear_sums_kernel(const PairArgs a, int64_t token_blocks) {
    constexpr int Q = kChunk<T>;
    const int tid = threadIdx.x;
    if ((int64_t)blockIdx.x >= token_blocks) {
        const int64_t h = blockIdx.x - token_blocks;
        double sum = 0.0;
        for (int64_t i = tid; i < a.items; i += 256) sum += a.skips[i * a.H + h];
        __shared__ double part[256];
        part[tid] = sum;
        __syncthreads();
        for (int d = 128; d; d >>= 1) {
            if (tid < d) part[tid] += part[tid + d];
            __syncthreads();
        }
        if (tid == 0) a.dD[h] = (float)part[0];
        return;
    }
    const int grp = (int)(blockIdx.x % a.G);
    Item it;
    if (!find_item(a.q, blockIdx.x / a.G, Q, it)) return;
    const int t0 = it.beg + it.c * Q, nt = min(Q, it.end - t0), N = (int)a.N;
    const int64_t all = a.Bsz * a.G * a.q.L * N;
    const float* from = a.parts + (((int64_t)it.row * a.G + grp) * a.q.L + t0) * N;
    const bool by_step = a.dq.sl == 1 && a.dk.sl == 1;
    for (int e = tid; e < nt * N; e += 256) {
        const int r = by_step ? e % nt : e / N, n = by_step ? e / nt : e % N;
        float q = 0.0f, k = 0.0f;
        for (int b = 0; b < a.blocks; ++b) {
            q += from[b * 2 * all + (int64_t)r * N + n];
            k += from[b * 2 * all + all + (int64_t)r * N + n];
        }
        ((T*)a.dq.data)[it.row * a.dq.sb + grp * a.dq.sg + (t0 + r) * a.dq.sl + n * a.dq.sn] = from_f<T>(q);
        ((T*)a.dk.data)[it.row * a.dk.sb + grp * a.dk.sg + (t0 + r) * a.dk.sl + n * a.dk.sn] = from_f<T>(k);
    }
}

template <class T>
hipError_t launch_pairs(const PairArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.items * a.G * a.blocks));
    if (a.N <= 32) hipLaunchKernelGGL((linear_pairs_kernel<T, 32>), grid, dim3(kPairThreads<32>), 0, s, a);
    else if (a.N <= 64) hipLaunchKernelGGL((linear_pairs_kernel<T, 64>), grid, dim3(kPairThreads<64>), 0, s, a);
    else if (a.N <= 128) hipLaunchKernelGGL((linear_pairs_kernel<T, 128>), grid, dim3(kPairThreads<128>), 0, s, a);
    else hipLaunchKernelGGL((linear_pairs_kernel<T, 256>), grid, dim3(kPairThreads<256>), 0, s, a);
    const int64_t tokens = a.blocks > 1 ? a.items * a.G : 0, heads = a.skips ? a.H : 0;
    if (tokens + heads)
        hipLaunchKernelGGL((linear_sums_kernel<T>), dim3((unsigned)(tokens + heads)), dim3(256), 0, s, a, tokens);
    return hipGetLastError();
}

}  // namespace ssm

// The gradients of linear attention's queries, keys, decays and weights
// (include/ssm.h: ssm_linear_attention_backward), from the states before every chunk and
// the gradients of the states behind them.
#pragma once

#include "linear.hpp"

namespace ssm {

constexpr int kPairValues = 64;
constexpr int kPairThreads = 512;

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
// float32 of float32 numbers: x and X are split (kParts); u beta dM, for dq and dk alone, is an
// operand in two parts (kShort).
// Values beyond 64 go block by block; every sum is linear in them.  q_t . k_s is formed
// once for all heads.  A wave has 16 keys (or more), and all steps or some of them; results
// lie transposed (lane: step, registers: four keys), so that rows of four keys are
// multiplied with q and k at once.  The sums over pairs and keys go through LDS and become dg
// and dbeta a block later, in the last wave, beside the other waves' pairs; so do the decays
// of the head after the next.
// 128 chunks of 64 steps, 64 heads of 128 keys and 64 values, one group, bf16: 240 us.  The saved
// states alone, 537 MB, take 113 us at a copy's rate; of the rest, vector instructions (a third
// of them split the states) and the tiles' reads from LDS have most, at two waves to a SIMD.
template <class T, int NP, bool FAST>
__global__ __launch_bounds__(kPairThreads, 2) void linear_pairs_kernel(const PairArgs a) {
    constexpr int TH = kPairThreads, W = TH / 64;
    constexpr int Q = kChunk<T>, TT = Q / 16, KK = NP / 32, SS = Q / 32, PK = kPairValues / 32;
    constexpr int TILES = NP / 16, NT = TILES > W ? TILES / W : 1;  // tiles of keys, and those of a wave
    constexpr int GROUPS = TILES >= W ? 1 : W / TILES < TT ? W / TILES : TT, TW = TT / GROUPS;  // of the steps; tiles of one
    constexpr int KS = NP + kRoom<T>, VS = kPairValues + kRoom<T>, K2 = kShort<T>;
    using Pairs = PairPlaces<T>;
    constexpr bool F16 = std::is_same<T, f16>::value;
    // The states of the next block are loaded a block ahead, and v and dy two, where the registers
    // and LDS take it.  In float32 two workgroups share a compute unit instead: 27 us at 256 chunks of
    // 32 steps, 4 heads of 64 keys and values in two groups; loaded ahead, with one workgroup, 36.
    constexpr bool EARLY = sizeof(T) == 2 && NT == 1;
    constexpr int RING = EARLY ? 3 : 2;  // tiles of v and dy
    struct PairSums {  // of W over the pairs of a tile's rows and columns, and on the diagonal
        float rows[TT][Q], columns[TT][Q], diagonal[Q], skip[TT];
    };
    constexpr int KEYS = TILES / NT;  // a wave's tiles are added up
    struct KeySums {
        float before[KEYS][Q], behind[KEYS][Q], whole[KEYS];
    };
    struct __attribute__((aligned(16))) Shared {
        T q[Q * KS], k[Q * KS], v[RING][Q * VS], dy[RING][Q * VS], m[2][K2 * Pairs::kSize];
        Decays<T> d[4];
        float beta[4][Q];
        float next[4], across[4], most_beta[4];  // the decay to the next chunk's first step; over the chunk and it
        PairSums pairs[3];
        KeySums keys[2];
        uint32_t most[2][2][W];
    };
    __shared__ Shared sh;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t bid = blockIdx.x;
    const int blk = (int)(bid % a.blocks), grp = (int)(bid / a.blocks % a.G);
    const int64_t item = bid / a.blocks / a.G;
    const int Hg = (int)(a.H / a.G), h0 = grp * Hg + blk * a.heads, h1 = min(h0 + a.heads, (grp + 1) * Hg);
    Item it;
    const bool found = find_item(a.q, item, Q, it);
    const int t0 = found ? it.beg + it.c * Q : 0, nt = found ? min(Q, it.end - t0) : 0;
    if (nt <= 0) {
        if (a.skips)
            for (int h = h0 + (int)threadIdx.x; h < h1; h += TH) a.skips[item * a.H + h] = 0.0f;
        return;
    }
    const int N = (int)a.N, P = (int)a.P, values = (P + kPairValues - 1) / kPairValues;
    const int Np = (int)padded_keys(a.N), Pp = (int)padded_values(a.P);
    const int64_t row = (linear_row(a.q, it, Q) + it.c) * a.H;

    {
        const int tid = threadIdx.x;
        Carrier<T, NP, TH, FAST> cq, ck;
        cq.load(a.qv.data + it.row * a.qv.sb + grp * a.qv.sg + t0 * a.qv.sl, a.qv, N, nt, tid);
        ck.load(a.k.data + it.row * a.k.sb + grp * a.k.sg + t0 * a.k.sl, a.k, N, nt, tid);
        cq.clear(a.qv.lay, N, nt, tid);
        ck.clear(a.k.lay, N, nt, tid);
        cq.template store<false>(sh.q, a.qv.lay, tid);
        ck.template store<false>(sh.k, a.k.lay, tid);
        for (int i = tid; i < 2 * K2 * Pairs::kSize; i += TH) sh.m[0][i] = from_f<T>(0.0f);  // pairs s > t stay zero
    }
    struct Block {  // of values of a head
        int h, pb;
    };
    Carrier<T, kPairValues, TH, FAST> cv, cy;
    auto load = [&](const Block& b) {
        const int h = b.h, p0 = b.pb * kPairValues, tid = threadIdx.x;
        cv.load(a.v.data + it.row * a.v.sb + h * a.v.sg + t0 * a.v.sl + p0 * a.v.sn, a.v, P - p0, nt, tid);
        cy.load(a.dy.data + it.row * a.dy.sb + h * a.dy.sg + t0 * a.dy.sl + p0 * a.dy.sn, a.dy, P - p0, nt, tid);
    };
    // the last wave: the decays of a head
    float g = 0.0f, beta = 0.0f, g_next = 0.0f;
    auto load_decays = [&](int h) {
        const int lane = threadIdx.x & 63;
        const float* gs = (const float*)a.g.data + it.row * a.g.sb + h * a.g.sh;
        g = beta = 0.0f;
        if (lane < nt) {
            g = gs[(t0 + lane) * a.g.sl];
            beta = a.beta.data ? ((const float*)a.beta.data)[it.row * a.beta.sb + h * a.beta.sh + (t0 + lane) * a.beta.sl] : 1.0f;
        }
        g_next = t0 + nt < it.end ? gs[(t0 + nt) * a.g.sl] : 0.0f;
    };
    auto keep_decays = [&](int i) {
        const int lane = anew(threadIdx.x) & 63;
        put_decays<T>(sh.d[i], g, lane < nt ? 1.0f : 0.0f, lane < nt ? a.scale : 0.0f, lane);
        if (lane < Q) sh.beta[i][lane] = beta;
        const float all = across_rows(row_sum(g));
        if (lane == 0) sh.across[i] = exp_f<kFine<T>>(all + g_next), sh.next[i] = exp_f<kFine<T>>(g_next);
        if constexpr (F16) {
            float m = fabsf(beta);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
            if (lane == 0) sh.most_beta[i] = m;
        }
    };
    // and, lane r, a head's sums over its blocks of values
    float sum_row = 0.0f, sum_column = 0.0f, sum_diagonal = 0.0f, sum_before = 0.0f, sum_behind = 0.0f, sum_whole = 0.0f,
          sum_skip = 0.0f;
    auto collect = [&](const PairSums& s, const KeySums& o) {
        const int lane = anew(threadIdx.x) & 63;
        if (lane < Q) {
            const int own = lane >> 4;
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                sum_row += i <= own ? s.rows[i][lane] : 0.0f;
                sum_column += i >= own ? s.columns[i][lane] : 0.0f;
            }
            sum_diagonal += s.diagonal[lane];
#pragma unroll
            for (int i = 0; i < KEYS; ++i) sum_before += o.before[i][lane], sum_behind += o.behind[i][lane];
        }
#pragma unroll
        for (int i = 0; i < KEYS; ++i) sum_whole += o.whole[i];
#pragma unroll
        for (int i = 0; i < TT; ++i) sum_skip += s.skip[i];
    };
    auto finish = [&](int h, int i) {  // of head h, whose decays are in place i
        const int lane = anew(threadIdx.x) & 63, r = min(lane, Q - 1);
        // (a weight of zero takes part in nothing, whatever its step's keys and values make of its sums)
        const float b = sh.beta[i][r], own = b == 0.0f ? 0.0f : b * sum_behind;
        // sums over the steps from r on, and before r
        float from = row_suffix(sum_row + sum_before - (b == 0.0f ? 0.0f : b * sum_column)), till = row_prefix(own);
        float later = 0.0f, earlier = 0.0f;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const float f = of_lane(from, 16 * i), e = of_lane(till, 16 * i + 15);
            later += i > (lane >> 4) ? f : 0.0f, earlier += i < (lane >> 4) ? e : 0.0f;
        }
        from += later, till += earlier;
        const float dg = from + (till - own) + (sh.across[i] == 0.0f ? 0.0f : sh.across[i] * sum_whole);
        if (lane < nt) {
            // a reset takes part in no product, and the sums' rounding is not left in its place
            ((float*)a.dg.data)[it.row * a.dg.sb + h * a.dg.sh + (t0 + lane) * a.dg.sl] =
                exp_f<kFine<T>>(sh.d[i].g[r]) == 0.0f ? 0.0f : dg;
            if (a.dbeta.data)
                ((float*)a.dbeta.data)[it.row * a.dbeta.sb + h * a.dbeta.sh + (t0 + lane) * a.dbeta.sl] =
                    sum_column + sum_diagonal + sum_behind;
        }
        if (a.skips && lane == 0) a.skips[item * a.H + h] = sum_skip;
        sum_row = sum_column = sum_diagonal = sum_before = sum_behind = sum_whole = sum_skip = 0.0f;
    };

    const int count = (h1 - h0) * values;
    auto behind = [&](const Block& b) { return b.pb + 1 == values ? Block{b.h + 1, 0} : Block{b.h, b.pb + 1}; };
    auto place = [&](int h) { return (h - h0) & 3; };  // of a head's decays
    // block k's tiles, loaded before
    auto store = [&](const Block& b, int k) {
        const int tid = threadIdx.x, i = k % RING;
        cv.clear(a.v.lay, P - b.pb * kPairValues, nt, tid);
        cy.clear(a.dy.lay, P - b.pb * kPairValues, nt, tid);
        cv.template store<false>(sh.v[i], a.v.lay, tid);
        cy.template store<false>(sh.dy[i], a.dy.lay, tid);
        if constexpr (F16) {
            uint32_t mv = cv.most(), my = cy.most();
#pragma unroll
            for (int i = 1; i < 64; i <<= 1)
                mv = max(mv, (uint32_t)__shfl_xor((int)mv, i)), my = max(my, (uint32_t)__shfl_xor((int)my, i));
            if ((tid & 63) == 0) sh.most[k & 1][0][wave] = mv, sh.most[k & 1][1][wave] = my;
        }
    };
    Block now = {h0, 0}, next = now;  // blocks k and k + 1
    load(next);
    if (wave == W - 1) {
        load_decays(h0);
        keep_decays(0);
        if (h0 + 1 < h1) load_decays(h0 + 1);
    }
    store(next, 0);
    if (count > 1) {
        const Block second = behind(next);
        load(second);
    }
    __syncthreads();

    // the wave's pairs: a tile on the diagonal, or one or two below it
    constexpr int BELOW = TT * (TT - 1) / 2, OWN = BELOW > 3 ? 2 : 1;
    auto below = [](int j, int& ti, int& si) {
        ti = j < 1 ? 1 : j < 3 ? 2 : 3;
        si = j - ti * (ti - 1) / 2;
    };
    const bool diagonal = wave < TT;
    const int first = diagonal ? 0 : wave < 4 || wave == W - 1 ? BELOW : wave - 4;  // (the last wave has the sums)
    f32x4 qk[OWN];
    uint32_t far_qk[OWN] = {};  // rows of keys and queries whose products are kept 2^-98 times
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        qk[j] = f32x4{0, 0, 0, 0};
        int ti = wave, si = wave;
        if (!diagonal) below(first + 3 * j, ti, si);
        if (diagonal ? j == 0 : first + 3 * j < BELOW) {
            const int lane = threadIdx.x & 63;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                qk[j] = mma<T>(row_frag<T>(sh.k + (16 * si + (lane & 15)) * KS + 32 * kk + 8 * (lane >> 4)),
                               row_frag<T>(sh.q + (16 * ti + (lane & 15)) * KS + 32 * kk + 8 * (lane >> 4)), qk[j]);
            const f32x4 one[1] = {qk[j]};
            if (!F16 && __builtin_expect(__ballot(far_out(one)) != 0, 0))
                qk[j] = products_in_range<T, KK>(sh.k + (16 * si + (lane & 15)) * KS + 8 * (lane >> 4),
                                                 sh.q + (16 * ti + (lane & 15)) * KS + 8 * (lane >> 4), far_qk[j]);
        }
    }
    // the wave's keys and steps
    const int tile = TILES >= W ? wave * NT : wave % TILES, n0 = 16 * tile, group = TILES >= W ? 0 : wave / TILES;
    const bool live = group < GROUPS;
    f32x4 dq[NT][TW], dk[NT][TW];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TW; ++t) dq[n][t] = dk[n][t] = f32x4{0, 0, 0, 0};

    // the states' fragments: keys n0 + 16 n + tl, values 32 kk + 8 gl .. + 7.  A block's are loaded
    // when the last one's have been used (EARLY).
    f32x4 x[PK][2], X[PK][2];
    auto load_states = [&](f32x4 (&to)[PK][2], const float* from, const Block& b, int n) {
        const int lane = anew(threadIdx.x) & 63;
        const float* at = from + (row + b.h) * Np * Pp + ((tile + n) * Pp + b.pb * kPairValues + 8 * (lane >> 4)) * 16 + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < PK; ++kk) {
            to[kk][0] = to[kk][1] = f32x4{0, 0, 0, 0};
            if (live && n0 + 16 * n < Np && b.pb * kPairValues + 32 * kk < Pp) {
#pragma unroll
                for (int i = 0; i < 8; ++i) to[kk][i / 4][i % 4] = at[(32 * kk + i) * 16];
            }
        }
    };
    if (EARLY) load_states(x, a.states, next, 0), load_states(X, a.ahead, next, 0);
    float sm = 1.0f;
    // Block k's keys beside block k + 1's pairs and block k + 2's way to LDS, with one barrier (or
    // two): with one block at a time, three barriers and the states loaded when they are needed,
    // 272 us instead of 259.
    for (int k = -1; k < count; ++k) {
        const int tid = anew(threadIdx.x), lane = tid & 63, tl = lane & 15, gl = lane >> 4;  // (addresses are not kept)
        const Block far = behind(next);
        auto take = [&]() {
            if (k + 2 >= count) return;
            store(far, k + 2);
            const Block last = behind(far);
            if (k + 3 < count) load(last);
        };
        if (RING > 2) take();
        if (k >= 0 && live) {  // keys by steps: dq and dk
            const Decays<T>& d = sh.d[place(now.h)];
            const T *v = sh.v[k % RING], *dy = sh.dy[k % RING], *m = sh.m[k & 1];
            KeySums& sums = sh.keys[k & 1];
            const float um = reciprocal_of_power(sm), further = sh.next[place(now.h)];
            // (added up over a wave's tiles in LDS, not in registers)
            auto keep = [&](float& to, float x, int n) { to = n ? to + x : x; };
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int key = n0 + 16 * n;
                if (!EARLY) load_states(x, a.states, now, n), load_states(X, a.ahead, now, n);
                float whole = 0.0f;
#pragma unroll
                for (int kk = 0; kk < PK; ++kk)
#pragma unroll
                    for (int i = 0; i < 8; ++i) whole = fmaf(x[kk][i / 4][i % 4], X[kk][i / 4][i % 4], whole);
                // products of the states with a tile of steps (dy or v), and what brings them back to scale
                auto across = [&](f32x4 (&state)[PK][2], const float* all, const T* tile, f32x4 (&to)[TW]) {
                    const int lane = anew(tid) & 63, tl = lane & 15, gl = lane >> 4;
                    float s = 1.0f;
                    if constexpr (F16) {
                        float m = 0.0f;
#pragma unroll
                        for (int kk = 0; kk < PK; ++kk)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float u = fabsf(state[kk][i / 4][i % 4]);
                                m = fmaxf(m, u < INFINITY ? u : 0.0f);
                            }
#pragma unroll
                        for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i));
                        s = to_range<T>(m);
                    }
                    while (true) {
#pragma unroll
                        for (int t = 0; t < TW; ++t) to[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int kk = 0; kk < PK; ++kk) {
                            float u[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) u[i] = F16 ? state[kk][i / 4][i % 4] * s : state[kk][i / 4][i % 4];
                            Frag<T> part[kParts<T>];
                            split<T>(u, part);
                            Frag<T> f[TW];
#pragma unroll
                            for (int t = 0; t < TW; ++t) f[t] = row_frag<T>(tile + (16 * (TW * group + t) + tl) * VS + 32 * kk + 8 * gl);
                            // (products that wait for each other's sums do not follow each other)
#pragma unroll
                            for (int i = 0; i < kParts<T>; ++i)
#pragma unroll
                                for (int t = 0; t < TW; ++t) to[t] = mma<T>(part[i], f[t], to[t]);
                        }
                        // (a state or a value so large that the products pass float32: once more, 2^-64 times,
                        // read again so that nothing is kept for it)
                        if (F16 || s != 1.0f || __builtin_expect(__ballot(far_out(to)) == 0, 1)) break;
                        s = 0x1p-64f;
                        load_states(state, all, now, n);
#pragma unroll
                        for (int kk = 0; kk < PK; ++kk) state[kk][0] *= s, state[kk][1] *= s;
                    }
                    return reciprocal_of_power(s);
                };
                struct __attribute__((aligned(4 * sizeof(T)))) Own { Quad<T> v; };
                {
                    const int lane = anew(tid) & 63, tl = lane & 15, gl = lane >> 4;
                    f32x4 in[TW];
                    const float ux = across(x, a.states, dy, in);
                    if (EARLY && k + 1 < count) load_states(x, a.states, next, 0);
                    Frag<T> kf[SS];
#pragma unroll
                    for (int s = 0; s < SS; ++s) kf[s] = column_frag<T>(sh.k + 32 * s * KS + key, KS, lane);
#pragma unroll
                    for (int t = 0; t < TW; ++t) {
                        const int tt = TW * group + t, r = 16 * tt + tl;
                        f32x4 w = {0, 0, 0, 0};
#pragma unroll
                        for (int i = K2 - 1; i >= 0; --i) {
#pragma unroll
                            for (int s = 0; s < SS; ++s)
                                if (s <= tt / 2)
                                    w = mma<T>(kf[s], row_frag<T>(m + Pairs::row(tt / 2, r) + i * Pairs::kSize + 32 * s + 8 * gl), w);
                            w *= i ? 1.0f / kLift<T> : 1.0f;
                        }
                        const float from = d.from[r];
                        const Own q4 = *reinterpret_cast<const Own*>(sh.q + r * KS + key + 4 * gl);
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = in[t][i] * from;
                            sum = fmaf(u, to_f(get_of<T>(q4.v, i)), sum);
                            dq[n][t][i] = fmaf(u, ux, fmaf(w[i], um, dq[n][t][i]));
                        }
                        sum = across_rows(sum) * ux;
                        if (gl == 0) keep(sums.before[tile / NT][r], sum, n);
                    }
                }
                {
                    const int lane = anew(tid) & 63, tl = lane & 15, gl = lane >> 4;
                    f32x4 out[TW];
                    const float uX = across(X, a.ahead, v, out);
                    if (EARLY && k + 1 < count) load_states(X, a.ahead, next, 0);
                    Frag<T> qf[SS];
#pragma unroll
                    for (int s = 0; s < SS; ++s) qf[s] = column_frag<T>(sh.q + 32 * s * KS + key, KS, lane);
#pragma unroll
                    for (int t = 0; t < TW; ++t) {
                        const int tt = TW * group + t, r = 16 * tt + tl;
                        f32x4 w = {0, 0, 0, 0};
#pragma unroll
                        for (int i = K2 - 1; i >= 0; --i) {
#pragma unroll
                            for (int s = 0; s < SS; ++s)
                                if (s >= tt / 2)
                                    w = mma<T>(qf[s], column_frag<T>(m + Pairs::row(s, 32 * s) + i * Pairs::kSize + 16 * tt, Pairs::stride(s), lane), w);
                            w *= i ? 1.0f / kLift<T> : 1.0f;
                        }
                        const float to = d.to[r] * further, b = sh.beta[place(now.h)][r] * uX;
                        const Own k4 = *reinterpret_cast<const Own*>(sh.k + r * KS + key + 4 * gl);
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = out[t][i] * to;
                            sum = fmaf(u, to_f(get_of<T>(k4.v, i)), sum);
                            dk[n][t][i] = fmaf(u, b, fmaf(w[i], um, dk[n][t][i]));
                        }
                        sum = across_rows(sum) * uX;
                        if (gl == 0) keep(sums.behind[tile / NT][r], sum, n);
                    }
                }
                whole = across_rows(row_sum(whole));
                if (lane == 0) keep(sums.whole[tile / NT], whole, n);
            }
        }
        if (k + 1 < count) {  // the pairs
            const Decays<T>& d = sh.d[place(next.h)];
            const T *v = sh.v[(k + 1) % RING], *dy = sh.dy[(k + 1) % RING];
            T* m = sh.m[(k + 1) & 1];
            PairSums& sums = sh.pairs[(k + 1) % 3];
            if constexpr (F16) {
                uint32_t mv = 0, my = 0;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    mv = max(mv, sh.most[(k + 1) & 1][0][i]), my = max(my, sh.most[(k + 1) & 1][1][i]);
                sm = to_range<T>(fabsf(a.scale) * d.grow * sh.most_beta[place(next.h)] * (float)kPairValues *
                                 to_f(__builtin_bit_cast(f16, (uint16_t)mv)) * to_f(__builtin_bit_cast(f16, (uint16_t)my)));
            }
            auto pairs = [&](int ti, int si, const f32x4& u, const f32x4& kq, uint32_t far_kq, bool on) {
                f32x4 dm = {0, 0, 0, 0};
                uint32_t far_dm = 0;
#pragma unroll
                for (int kk = 0; kk < PK; ++kk)
                    dm = mma<T>(row_frag<T>(v + (16 * si + tl) * VS + 32 * kk + 8 * gl),
                                row_frag<T>(dy + (16 * ti + tl) * VS + 32 * kk + 8 * gl), dm);
                const f32x4 one[1] = {dm};
                if (!F16 && __builtin_expect(__ballot(far_out(one)) != 0, 0))
                    dm = products_in_range<T, PK>(v + (16 * si + tl) * VS + 8 * gl, dy + (16 * ti + tl) * VS + 8 * gl, far_dm);
                const f32x4 b = *reinterpret_cast<const f32x4*>(&sh.beta[place(next.h)][16 * si + 4 * gl]);
                f32x4 w;
                float column[4], part = 0.0f, skip = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool own = on && 4 * gl + i == tl;
                    const float um = u[i] * dm[i];
                    float wt = um * kq[i], ub = um * b[i], wb = ub * kq[i], yv = dm[i];
                    if (__builtin_expect((far_kq | far_dm) != 0, 0)) {
                        auto product = [&](float x) {
                            float y = kq[i];
                            bring_back(x, y, far_dm, 4 * gl + i, tl);
                            bring_back(x, y, far_kq, 4 * gl + i, tl);
                            return x * y;
                        };
                        float one = 1.0f;
                        wt = product(um), wb = product(ub);
                        bring_back(ub, one, far_dm, 4 * gl + i, tl), ub *= one, one = 1.0f;
                        bring_back(yv, one, far_dm, 4 * gl + i, tl), yv *= one;
                        // a value that nothing is to be weighted with must not make an infinity of that
                        if (kq[i] == 0.0f && fabsf(um) < INFINITY) ub = fminf(fmaxf(ub, -kLargest<T>), kLargest<T>);
                    }
                    if (own) sums.diagonal[16 * ti + tl] = wt;
                    column[i] = own ? 0.0f : wt;
                    skip = own ? yv : skip;
                    part += own ? 0.0f : wb;
                    w[i] = ub * sm;
                }
                put_parts<T, K2>(m + Pairs::row(ti >> 1, 16 * ti + tl) + 16 * si + 4 * gl, Pairs::kSize, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) column[i] = row_sum(column[i]);
                if (tl == 0)
                    *reinterpret_cast<f32x4*>(&sums.columns[ti][16 * si + 4 * gl]) = f32x4{column[0], column[1], column[2], column[3]};
                part = across_rows(part);
                if (gl == 0) sums.rows[si][16 * ti + tl] = part;
                if (on) {
                    skip = across_rows(row_sum(skip));
                    if (lane == 0) sums.skip[ti] = skip;
                }
            };
            if (diagonal) {
                pairs(wave, wave, weights_within<T>(d, wave, lane), qk[0], far_qk[0], true);
            } else {
#pragma unroll
                for (int j = 0; j < OWN; ++j) {
                    int ti, si;
                    below(first + 3 * j, ti, si);
                    if (first + 3 * j < BELOW) pairs(ti, si, weights_across<T>(d, ti, si, lane), qk[j], far_qk[j], false);
                }
            }
        }
        if (wave == W - 1) {
            if (k > 0) {
                collect(sh.pairs[(k - 1) % 3], sh.keys[(k - 1) & 1]);
                if (now.pb == 0) finish(now.h - 1, place(now.h - 1));
            }
            if (far.h > next.h && far.h < h1) {
                keep_decays(place(far.h));
                if (far.h + 1 < h1) load_decays(far.h + 1);
            }
        }
        __syncthreads();
        if (RING == 2) {
            take();
            __syncthreads();
        }
        now = next, next = far;
    }
    if (wave == W - 1) {
        collect(sh.pairs[(count - 1) % 3], sh.keys[(count - 1) & 1]);
        finish(h1 - 1, place(h1 - 1));
    }
    if (!live) return;
    const int lane = anew(threadIdx.x) & 63, tl = lane & 15, gl = lane >> 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            const int r = 16 * (TW * group + t) + tl, key = n0 + 16 * n + 4 * gl, there = N - key;
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
    constexpr int R = 8;  // steps of a workgroup
    const int64_t part = blockIdx.x / a.G;
    Item it;
    if (!find_item(a.q, part / (Q / R), Q, it)) return;
    const int t0 = it.beg + it.c * Q + (int)(part % (Q / R)) * R, nt = min(R, it.end - t0), N = (int)a.N;
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

template <class T, int NP>
static void launch_pairs_keys(const PairArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.items * a.G * a.blocks)), wg(kPairThreads);
    if (a.fast) hipLaunchKernelGGL((linear_pairs_kernel<T, NP, true>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((linear_pairs_kernel<T, NP, false>), grid, wg, 0, s, a);
}
template <class T>
hipError_t launch_pairs(const PairArgs& a, hipStream_t s) {
    if (a.N <= 32) launch_pairs_keys<T, 32>(a, s);
    else if (a.N <= 64) launch_pairs_keys<T, 64>(a, s);
    else if (a.N <= 128) launch_pairs_keys<T, 128>(a, s);
    else launch_pairs_keys<T, 256>(a, s);
    const int64_t tokens = a.blocks > 1 ? a.items * (kChunk<T> / 8) * a.G : 0, heads = a.skips ? a.H : 0;
    if (tokens + heads)
        hipLaunchKernelGGL((linear_sums_kernel<T>), dim3((unsigned)(tokens + heads)), dim3(256), 0, s, a, tokens);
    return hipGetLastError();
}

}  // namespace ssm

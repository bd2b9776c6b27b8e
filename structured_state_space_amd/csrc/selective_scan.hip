// Selective state-space scan, forward:
//   dt = softplus(delta + delta_bias)
//   x_t[n] = exp(dt_t A[n]) x_{t-1}[n] + dt_t u_t B_t[n]
//   y_t = (sum_n C_t[n] x_t[n] + D u_t) silu(z_t)
// per (sequence, channel), B and C shared by the channels of a group.
//
// Work split.  A workgroup has 64 channels of one group and takes the steps in
// order, 32 to a tile: its threads move a tile's elements in vectors, prepare them
// (softplus) and leave dt and dt u in LDS; then eight lanes per channel run the
// recurrence, B and C in LDS too, and leave their sums for y there; then the movers
// apply skip term and gate.  The next tile's loads fly while one is run.
//
// Where channels and sequences alone leave the GPU idle, the steps are split
// into chunks of Q as well: a first launch computes every chunk's state from a
// zero start (without C and y) and the sum of its dt, whose exp(A sum dt) is
// the chunk's whole decay; in the second each chunk folds its predecessors'
// ends into its start state and runs the full recurrence.
//
// The vector ALU bounds it: a step of a state is a product, an exponential (a
// quarter of the rate), a product and two multiply-adds, 8.3 instructions with the
// moving and the sums over lanes.  bf16, N = 16, with gate: 1 row of 2048 channels x
// 16384 steps 106 us for the ends and 163 for the rest, vector instructions issuing in
// 97% of the busy cycles, 1.7 TB/s; 4 x 4096 x 2048 with its states saved, one workgroup
// per CU, 192 us, 76%.  With N = 17 to 32, any strides (float32: by tokens too) keep 12
// to 24 bytes a lane in scratch.
// (Both launches of the first case, call for call: 332 us with four lanes per
// channel, 308 with eight whose lanes loaded their own channels' steps, 280 with
// the roles apart, 235 with LDS layouts off each other's banks and 32-bit distances.)
#include "selective.hpp"

namespace ssm {

namespace {

// one tile's recurrence; GUARD: only the first nt steps exist (a branch per step), and
// the lane's states from the real-th on are held at zero (where dt and dt u are finite,
// they stay so by themselves).
// `bc` is the lane's B and C of the tile, `step` its channel's {dt, dt u}; both come
// from LDS two steps ahead of their use.
template <int S, bool ENDS, bool GUARD>
__device__ __forceinline__ void run_tile(float (&h)[S], const float (&A2)[S], const float* bc, const float* step,
                                         int nt, int real, float* ysum, int c, int p) {
    constexpr int kRow = Stage<float, S>::kRow, kGroup = S == 2 ? 2 : 1;
    const bool odd = p & 1, high = p & 2;
    float4 v[2][kGroup][S / 2];
    float2 d[2][kGroup];
    float share[4];  // the lane's shares of y of four steps
    auto fetch = [&](int g) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            d[g & 1][i] = *reinterpret_cast<const float2*>(step + (g * kGroup + i) * kPairRow);
#pragma unroll
            for (int k = 0; k < S / 2; ++k)
                v[g & 1][i][k] = *reinterpret_cast<const float4*>(bc + (g * kGroup + i) * kRow + k * 32);
        }
    };
    fetch(0);
#pragma unroll
    for (int g = 0; g < kTile / kGroup; ++g) {
        if (g + 1 < kTile / kGroup) fetch(g + 1);
        if (!GUARD) __builtin_amdgcn_sched_barrier(0);  // issue these reads before the steps below
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int t = g * kGroup + i;
            float acc = 0.0f;
            if (!GUARD || t < nt) {
                const float dt = d[g & 1][i].x, dx = d[g & 1][i].y;
#pragma unroll
                for (int k = 0; k < S / 2; ++k) {
                    const float4 w = v[g & 1][i][k];
                    h[2 * k] = fmaf(__builtin_amdgcn_exp2f(dt * A2[2 * k]), h[2 * k], dx * w.x);
                    h[2 * k + 1] = fmaf(__builtin_amdgcn_exp2f(dt * A2[2 * k + 1]), h[2 * k + 1], dx * w.y);
                    if (GUARD && !ENDS) {
                        h[2 * k] = 2 * k < real ? h[2 * k] : 0.0f;
                        h[2 * k + 1] = 2 * k + 1 < real ? h[2 * k + 1] : 0.0f;
                    }
                    if (!ENDS) acc = fmaf(w.w, h[2 * k + 1], k ? fmaf(w.z, h[2 * k], acc) : w.z * h[2 * k]);
                }
                // the sum is done here: left alone, the compiler moves the sums of the two
                // forms of this loop behind both of them and holds every step's states
                if (!ENDS) asm volatile("" : "+v"(acc));
            }
            share[t & 3] = acc;
            if (!ENDS && (t & 3) == 3)
                put_sums(ysum, t >> 2, quad_sums(share[0], share[1], share[2], share[3], odd, high), c, p);
        }
    }
}

struct Split {
    int Q;            // steps per chunk, a multiple of the tile
    int blocks;       // channel blocks
    int per_group;    // channel blocks of a group
    float* ends;      // [items, H, Np]: state at a chunk's end (chunk 0 from the initial state, others from 0)
    float* sums;      // [items, H]: sum of dt over a chunk
    float* starts;    // [S, H, Np]: copy of the initial states (x_out may be x_in)
};

// ENDS: the first launch of a split call, every chunk's end state and sum of dt
template <class T, int S, Order O, bool ENDS>
__global__ __launch_bounds__(kScanThreads, S <= 4 ? 4 : 2) void scan_kernel(ScanArgs a, Split sp) {
    constexpr int kRow = Stage<T, S>::kRow;
    __shared__ __attribute__((aligned(16))) float lds[kTile * kRow];
    __shared__ __attribute__((aligned(16))) float steps[kTile * kPairRow];
    __shared__ __attribute__((aligned(16))) float ysum[ENDS ? 4 : kTile * kPairRow];
    // an infinite or NaN dt u has come: its product with a padded state's B of zero is NaN,
    // which the sum over states would take for the channel's.  From that tile on the
    // guarded form runs, which holds padded states at zero (held in every tile, they
    // would cost two of 17 instructions per step); watching for it costs 1 to 2% with
    // padded states, nothing without.
    __shared__ int beyond;

    const int cb = blockIdx.x % sp.blocks;
    const int64_t item = blockIdx.x / sp.blocks;
    Item it;
    if (!find_item(a.q, item, sp.Q, it) || it.state < 0) return;
    const int64_t beg = it.beg + (int64_t)it.c * sp.Q;
    const int64_t end = min((int64_t)it.end, beg + sp.Q);
    const int chunks = chunks_of(it.end - it.beg, sp.Q);
    if (it.c >= chunks || (ENDS && it.c + 1 == chunks)) return;

    const Place l = place_of(cb, sp.per_group, a.H, a.G);
    const Mover<O> m(l.tid, l.valid);
    const int p = l.p, N = (int)a.N, real = N - p * S;
    const bool padded = N != 8 * S;  // some lanes have states that do not exist
    float A2[S], h[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        // behind the last state nothing decays or grows, whatever the sign of dt
        A2[j] = p * S + j < N ? a.A[(int64_t)l.h * N + p * S + j] * kLog2e : 0.0f;
        h[j] = 0.0f;
    }
    const int64_t wrow = (int64_t)l.h * (8 * S) + p * S;  // in a workspace row [H, Np]
    const int64_t wstep = a.H * (8 * S);

    if (!ENDS && padded) {
        if (l.tid == 0) beyond = 0;
        __syncthreads();
    }

    // start state
    if (it.c == 0) {
        if (!ENDS && sp.starts && chunks > 1) {
            load_states<S>(h, sp.starts + it.s * wstep + wrow);
        } else if (a.x_in) {
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (p * S + j < N) h[j] = a.x_in[(it.state * a.H + l.h) * N + p * S + j];
        }
        if (ENDS && l.live) store_states<S>(h, sp.starts + it.s * wstep + wrow);
    } else if (!ENDS) {
        const int64_t first = item - it.c;
        load_states<S>(h, sp.ends + first * wstep + wrow);
        for (int64_t i = first + 1; i < item; ++i) {
            const float s = sp.sums[i * a.H + l.h];
            float e[S];
            load_states<S>(e, sp.ends + i * wstep + wrow);
            over_chunk<S>(h, s, A2, e);
        }
        if (padded) {
#pragma unroll
            for (int j = 0; j < S; ++j) h[j] = j < real ? h[j] : 0.0f;
        }
    }

    const bool gate = !ENDS && a.z.data;
    const View3& gv = gate ? a.z : a.u;  // without a gate u once more, unused: the loads need no branch
    T ur[kOwn], dr[kOwn], zr[kOwn];
    const char* up = m.template base<T>(a.u, it.row, l, beg);
    const char* dp = m.template base<T>(a.delta, it.row, l, beg);
    const char* zp = m.template base<T>(gv, it.row, l, beg);
    char* yp = m.template base<T>(a.y, it.row, l, beg);
    const uint32_t uo = m.template offset<T>(a.u), dof = m.template offset<T>(a.delta),
                   zo = m.template offset<T>(gv), yo = m.template offset<T>(a.y);
    const char* Bp = group_base<T>(a.B, it.row, l.g, beg);
    const char* Cp = group_base<T>(a.C, it.row, l.g, beg);
    const Stage<T, S> stage(a.B, a.C, N, l.tid);
    T sb[Stage<T, S>::K], sc[Stage<T, S>::K];
    auto advance = [&](int64_t steps_on) {
        const int64_t e = steps_on * (int64_t)sizeof(T);
        up += e * a.u.sl, dp += e * a.delta.sl, zp += e * gv.sl, Bp += e * a.B.sl, Cp += e * a.C.sl;
    };
    auto load_tile = [&]() {
        m.template load<T>(ur, up, uo, a.u);
        m.template load<T>(dr, dp, dof, a.delta);
        if (!ENDS) m.template load<T>(zr, zp, zo, gv);
        stage.template load<true, !ENDS>(sb, sc, Bp, Cp);
    };
    float bias[kOwn], Dv[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int64_t hh = l.first + min(max(m.channel(i), 0), l.valid - 1);
        bias[i] = a.delta_bias ? a.delta_bias[hh] : 0.0f;
        Dv[i] = a.D ? a.D[hh] : 0.0f;
    }

    float uf[kOwn], zf[kOwn], sum[kOwn] = {};
    auto prepare = [&](int nt) {  // the loaded tile into LDS
        float d[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            uf[i] = to_f(ur[i]);
            if (!ENDS) zf[i] = to_f(zr[i]);
            d[i] = to_f(dr[i]) + bias[i];
        }
        if (a.softplus) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) d[i] = softplus_f<kFine<T>>(d[i]);
        }
        float dx[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (ENDS) sum[i] += m.step(i) < nt ? d[i] : 0.0f;
            dx[i] = d[i] * uf[i];
        }
        if (!ENDS && padded) {
            bool in = true;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) in = in && fabsf(dx[i]) < __builtin_inff();
            if (!in) beyond = 1;
        }
        put_pairs<O>(steps, d, dx, m, l.valid);
        stage.template store<true, !ENDS>(sb, sc, lds, nt);
        __syncthreads();
    };
    auto finish = [&](int nt) {  // y of the tile
        float yv[kOwn];
        get_sums<O>(yv, ysum, m);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) yv[i] = fmaf(Dv[i], uf[i], yv[i]);
        if (gate) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) yv[i] *= silu_f<kFine<T>>(zf[i]);
        }
        if (a.y.data) m.template store<T>(yv, yp, yo, a.y, l.valid, nt);
    };

    float* saved = !ENDS && a.saved && l.live
                       ? a.saved + (saved_row(a.q, it) + (beg - it.beg) / kTile) * wstep + wrow
                       : nullptr;
    const int len = (int)max((int64_t)0, end - beg), whole = len / kTile;
    int k = 0;
    if (whole > 0) load_tile();
    for (; k < whole; ++k) {
        prepare(kTile);
        if (!ENDS && padded && __builtin_amdgcn_readfirstlane(beyond)) break;
        // the next whole tile's loads fly while this one is run (the last one loads
        // itself again: a branch here would make them wait)
        advance(k + 1 < whole ? kTile : 0);
        load_tile();
        __builtin_amdgcn_sched_barrier(0);  // left alone, the compiler moves the loads behind the tile
        if (saved) {
            store_states<S>(h, saved);
            saved += wstep;
        }
        run_tile<S, ENDS, false>(h, A2, lds + p * 4, steps + pair_at(l.c), kTile, real, ysum, l.c, p);
        __syncthreads();
        if (!ENDS) finish(kTile);
        yp += kTile * a.y.sl * (int64_t)sizeof(T);
    }
    // the steps behind the last whole tile, and the tile left above with all behind it
    for (bool on = k == whole && whole > 0; k * kTile < len; ++k, on = true) {
        const int nt = min(kTile, len - k * kTile);
        advance(on ? kTile : 0);
        m.template load_part<T>(ur, up, uo, a.u, nt);
        m.template load_part<T>(dr, dp, dof, a.delta, nt);
        if (!ENDS) m.template load_part<T>(zr, zp, zo, gv, nt);
        stage.template load_part<true, !ENDS>(sb, sc, a.B, a.C, Bp, Cp, nt);
        prepare(nt);
        if (saved) {
            store_states<S>(h, saved);
            saved += wstep;
        }
        run_tile<S, ENDS, true>(h, A2, lds + p * 4, steps + pair_at(l.c), nt, real, ysum, l.c, p);
        __syncthreads();
        if (!ENDS) finish(nt);
        yp += kTile * a.y.sl * (int64_t)sizeof(T);
    }

    if (ENDS) {
        if (l.live) store_states<S>(h, sp.ends + item * wstep + wrow);
        // the channels' sums of dt, over the threads that moved their steps
        __syncthreads();
        float* const part = steps;
        constexpr int kParts = O == kRows ? 8 : kTile;
#pragma unroll
        for (int i = 1; i < (O == kRows ? kOwn : 1); ++i) sum[0] += sum[i];
#pragma unroll
        for (int i = 0; i < (O == kRows ? 1 : kOwn); ++i)
            if (m.has(i, l.valid)) part[(O == kRows ? l.tid & 7 : m.t) * kChannels + m.channel(i)] = sum[i];
        __syncthreads();
        if (l.tid < l.valid) {
            float s = 0.0f;
            for (int k = 0; k < kParts; ++k) s += part[k * kChannels + l.tid];
            sp.sums[item * a.H + l.first + l.tid] = s;
        }
    } else if (l.live && a.x_out && it.c + 1 == chunks) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (p * S + j < N) a.x_out[(it.state * a.H + l.h) * N + p * S + j] = h[j];
    }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
    Split sp;
    int64_t items;
    bool split;
    size_t ends_bytes, sums_bytes, starts_bytes;
};

Plan plan(const Seqs& q, int64_t H, int64_t N, int64_t G) {
    Plan p;
    const int64_t Hg = H / G;
    p.sp.per_group = (int)((Hg + kChannels - 1) / kChannels);
    p.sp.blocks = (int)(G * p.sp.per_group);
    const int64_t Q = chunk_steps(q, p.sp.blocks, N > 32 ? 4 : 3);
    p.sp.Q = (int)Q;
    p.split = Q < q.L;
    p.items = item_count(q, Q);
    const size_t Np = (size_t)padded_states(N);
    p.ends_bytes = p.split ? up256((size_t)p.items * H * Np * 4) : 0;
    p.sums_bytes = p.split ? up256((size_t)p.items * H * 4) : 0;
    p.starts_bytes = p.split ? up256((size_t)q.S * H * Np * 4) : 0;
    return p;
}

template <class T, int S, Order O>
hipError_t launch_as(const ScanArgs& a, const Plan& p, hipStream_t s) {
    const int64_t wgs = p.items * p.sp.blocks;
    if (!grid_fits(wgs, kScanThreads)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), wg(kScanThreads);
    if (p.split) scan_kernel<T, S, O, true><<<grid, wg, 0, s>>>(a, p.sp);
    scan_kernel<T, S, O, false><<<grid, wg, 0, s>>>(a, p.sp);
    return hipGetLastError();
}

template <class T, int S>
hipError_t launch_in(const ScanArgs& a, const Plan& p, Order o, hipStream_t s) {
    return o == kRows ? launch_as<T, S, kRows>(a, p, s)
         : o == kTokens ? launch_as<T, S, kTokens>(a, p, s) : launch_as<T, S, kAny>(a, p, s);
}

template <class T>
hipError_t launch_of(const ScanArgs& a, const Plan& p, Order o, hipStream_t s) {
    if (a.N <= 16) return launch_in<T, 2>(a, p, o, s);
    if (a.N <= 32) return launch_in<T, 4>(a, p, o, s);
    return launch_in<T, 8>(a, p, o, s);
}

}  // namespace

size_t scan_workspace_bytes(const Seqs& q, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, H, N, G);
    return p.ends_bytes + p.sums_bytes + p.starts_bytes;
}

bool scan_fits(const Seqs& q, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, H, N, G);
    return grid_fits(p.items * p.sp.blocks, kScanThreads);
}

hipError_t launch_scan(int dtype, const ScanArgs& a, void* ws, hipStream_t s) {
    Plan p = plan(a.q, a.H, a.N, a.G);
    if (p.split) {
        p.sp.ends = (float*)ws;
        p.sp.sums = (float*)((char*)ws + p.ends_bytes);
        p.sp.starts = (float*)((char*)ws + p.ends_bytes + p.sums_bytes);
    } else {
        p.sp.ends = p.sp.sums = p.sp.starts = nullptr;
    }
    const View3* views[] = {&a.u, &a.delta, &a.z, &a.y};
    const Order o = order_of(views, 4, a.H / a.G);
    if (dtype == SSM_F32) return launch_of<float>(a, p, o, s);
    if (dtype == SSM_BF16) return launch_of<bf16>(a, p, o, s);
    return launch_of<f16>(a, p, o, s);
}

}  // namespace ssm

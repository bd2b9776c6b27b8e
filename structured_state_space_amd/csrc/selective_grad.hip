// Selective state-space scan, backward.  With a_t = exp(dt_t A), the gate's
// gradient taken first (p_t = dy_t silu(z_t)) and, backwards in time,
//   g_t = C_t p_t + a_{t+1} g_{t+1}          (g behind the last step: dx_out)
// the gradients are
//   dB_t = sum_h g_t dt_t u_t        dC_t = sum_h p_t x_t
//   du_t = D p_t + dt_t sum_n g_t B_t
//   ddt_t = sum_n A a_t g_t x_{t-1} + u_t sum_n g_t B_t,  ddelta = ddt softplus'
//   dA = sum_{b,t} dt_t a_t g_t x_{t-1}   dD = sum p_t u_t   ddelta_bias = sum ddelta
//   dz_t = dy_t (sum_n C_t x_t + D u_t) silu'(z_t)          dx_in = a_1 g_1
//
// Work split as in the forward scan: 64 channels per workgroup, tiles of 32 steps,
// threads that move elements and eight lanes per channel that run the recurrence,
// LDS between them.  The tiles go from the last to the first: a tile's states are
// recomputed from the one that the forward pass saved at its first step (states
// and decays stay in registers, for one pair of a lane's states at a time), then
// the lanes walk back through it.
//
// dB and dC are sums over all channels of a group: over a wave's 8 channels by
// lane exchanges, over the workgroup's waves through LDS, over the group's
// workgroups by a second launch from one row of partial sums per workgroup.
// dA, dD and ddelta_bias are kept in registers over a workgroup's steps, and
// one row per workgroup is summed in float64.  Every order is fixed: a repeated
// call gives the same bits.
//
// Chunks of the steps, where channels and sequences are few, work as in the
// forward scan but from the end: a first launch gives each chunk's gradient
// towards the chunk before it from a zero end.
//
// The vector ALU bounds it: 27 instructions per step and state, of which the two
// walks take 20, the sums over lanes included, and moving the elements the rest.  bf16,
// N = 16, with gate, 4 x 4096 x 2048: 590 us and 18 for the last launch, vector
// instructions issuing in 76% of the busy cycles at one workgroup (146 KB of LDS, 208
// to 256 registers, two waves per SIMD) per CU, 0.75 TB/s.  What does not fit there: 21
// to 49 scalars lie in vector registers, and with N > 32 some forms keep 8 to 36 bytes a
// lane in scratch.  float32, N = 64, 8 x 256 x 1024 by rows: 37 us for the ends, 134,
// and 17.
#include "selective.hpp"

namespace ssm {

namespace {

// sums over the 8 channels of a wave (lane bits 3..5) of four values per lane, but
// for the last addition: lane l gets, of its lane position's value number l >> 4,
// what the channels with its bit 3 have
__device__ __forceinline__ float channel_sums(float v0, float v1, float v2, float v3) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v0), __float_as_uint(v2), false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v1), __float_as_uint(v3), false, false);
    const float x = __uint_as_float(a[0]) + __uint_as_float(a[1]);  // v0 below lane 32, v2 above
    const float y = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(c[0]) + __uint_as_float(c[1]);
}
// that addition for two steps' values: the first's for lanes with bit 3 clear, the second's for the others
__device__ __forceinline__ float last_sums(float first, float second, bool bit3) {
    return (bit3 ? second : first) + dpp<0x128>(bit3 ? first : second);  // row_ror:8
}

struct GradSplit {
    int Q, blocks, per_group;
    int64_t items;  // work items launched
    float* ends;    // [items, H, Np]: gradient a chunk hands to the chunk before it, from a zero end
    float* sums;    // [items, H]: sum of dt over a chunk
    float* part_bc; // [per_group, Bsz, L, G, S/2, 2, 16]: a workgroup's dB and dC by pairs of lane states
    float* part;    // [items, part_cols]: dA [H, Np], dD [H], ddelta_bias [H]
};
__host__ __device__ inline int64_t part_cols(int64_t H, int64_t Np) { return (H * (Np + 2) + 3) & ~(int64_t)3; }

// a row of `steps`: a place free behind every fourth channel, as in the rows of pairs
constexpr int kStepRow = kChannels / 4 * 5;
__device__ __forceinline__ int step_at(int c) { return c + (c >> 2); }

// ENDS: the first launch of a split call, what every chunk hands to the one before it
template <class T, int S, Order O, bool ENDS>
__global__ __launch_bounds__(kScanThreads, 2) void grad_kernel(ScanGradArgs ga, GradSplit sp) {
    const ScanArgs& a = ga.f;
    constexpr int kRow = Stage<T, S>::kRow;
    __shared__ __attribute__((aligned(16))) float lds[kTile * kRow];
    // {dt, dt u, p, slope of softplus} of every step and channel; p is the gradient behind the gate
    __shared__ __attribute__((aligned(16))) float4 steps[kTile * kStepRow];
    // sums over a channel's states: of C x, of g B, of A a g x
    __shared__ __attribute__((aligned(16))) float ysum[ENDS ? 4 : kTile * kPairRow];
    __shared__ __attribute__((aligned(16))) float gsum[ENDS ? 4 : kTile * kPairRow];
    __shared__ __attribute__((aligned(16))) float asum[ENDS ? 4 : kTile * kPairRow];
    __shared__ float red[ENDS ? 1 : 8 * kTile * 32];  // [wave][step][B or C][16 states]: sums over a wave's channels

    __shared__ float2 par[kChannels];  // {delta_bias, D}

    const int cb = blockIdx.x % sp.blocks;
    const int64_t item = blockIdx.x / sp.blocks;
    Item it;
    const bool there = find_item(a.q, item, sp.Q, it);
    const Place l = place_of(cb, sp.per_group, a.H, a.G);
    const Mover<O> m(l.tid, l.valid);
    const int p = l.p, N = (int)a.N, lane = l.tid & 63;
    const bool odd = p & 1, high = p & 2, bit3 = lane & 8;
    const int64_t wrow = (int64_t)l.h * (8 * S) + p * S, wstep = a.H * (8 * S);

    float A2[S], carry[S], dA[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        // behind the last state nothing decays or grows, whatever the sign of dt
        A2[j] = p * S + j < N ? a.A[(int64_t)l.h * N + p * S + j] * kLog2e : 0.0f;
        carry[j] = dA[j] = 0.0f;
    }
    float dDsum[kOwn] = {}, dbsum[kOwn] = {}, dtsum[kOwn] = {};

    const int chunks = there ? chunks_of(it.end - it.beg, sp.Q) : 0;
    const int64_t beg = there ? it.beg + (int64_t)it.c * sp.Q : 0;
    const int64_t end = there ? min((int64_t)it.end, beg + sp.Q) : 0;
    const bool work = there && it.c < chunks && (!ENDS || it.c > 0);
    if (ENDS && !work) return;
    if (work) {
        // the gradient that the steps behind this chunk hand to its last state;
        // lanes without a channel keep zero, and so add nothing to dB and dC
        if (it.c + 1 == chunks) {
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (ga.dx_out && l.live && p * S + j < N)
                    carry[j] = ga.dx_out[((int64_t)it.s * a.H + l.h) * N + p * S + j];
        } else if (!ENDS && l.live) {
            // (descending offsets may name more items than there are)
            const int64_t from = min(item + (chunks - 1 - it.c), sp.items - 1);
            if (from > item) load_states<S>(carry, sp.ends + from * wstep + wrow);  // with dx_out's part
            for (int64_t i = from - 1; i > item; --i) {
                const float s = sp.sums[i * a.H + l.h];
                float e[S];
                load_states<S>(e, sp.ends + i * wstep + wrow);
                over_chunk<S>(carry, s, A2, e);
            }
        }
    }

    if (work && beg < end) {
        const int tiles = (int)((end - beg + kTile - 1) / kTile);
        const int64_t last = beg + (int64_t)(tiles - 1) * kTile;  // the last tile's first step
        int now = (int)(end - last);                              // and its steps; all others are whole
        const bool gate = a.z.data;
        const View3& gv = gate ? a.z : a.u;  // without a gate u once more, unused
        const char* up = m.template base<T>(a.u, it.row, l, last);
        const char* dp = m.template base<T>(a.delta, it.row, l, last);
        const char* zp = m.template base<T>(gv, it.row, l, last);
        const char* gp = m.template base<T>(ga.dy, it.row, l, last);
        char* dup = m.template base<T>(ga.du, it.row, l, last);
        char* ddp = m.template base<T>(ga.ddelta, it.row, l, last);
        char* dzp = m.template base<T>(ga.dz, it.row, l, last);
        const char* Bp = group_base<T>(a.B, it.row, l.g, last);
        const char* Cp = group_base<T>(a.C, it.row, l.g, last);
        T sb[Stage<T, S>::K], sc[Stage<T, S>::K];
        const float* sv = ENDS ? nullptr : ga.saved + (saved_row(a.q, it) + (last - it.beg) / kTile) * wstep + wrow;
        if (l.tid < kChannels) {  // (in registers they would take eight)
            const int64_t hh = l.first + min(l.tid, l.valid - 1);
            par[l.tid] = make_float2(a.delta_bias ? a.delta_bias[hh] : 0.0f, a.D ? a.D[hh] : 0.0f);
        }
        __syncthreads();
        if (l.valid < kChannels) {  // channels that are not there: steps of length zero without gradient
            for (int e = l.tid; e < kTile * kStepRow; e += kScanThreads) steps[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            __syncthreads();
        }

        T ur[kOwn], dr[kOwn], zr[kOwn], gr[kOwn];
        float hn[S];
        m.template load_part<T>(ur, up, m.template offset<T>(a.u), a.u, now);
        m.template load_part<T>(dr, dp, m.template offset<T>(a.delta), a.delta, now);
        m.template load_part<T>(gr, gp, m.template offset<T>(ga.dy), ga.dy, now);
        m.template load_part<T>(zr, zp, m.template offset<T>(gv), gv, now);
        Stage<T, S>(a.B, a.C, N, l.tid).template load_part<!ENDS, true>(sb, sc, a.B, a.C, Bp, Cp, now);
        if (!ENDS) load_states<S>(hn, sv);

        for (int tile = tiles - 1; tile >= 0; --tile) {
            const int64_t t0 = beg + (int64_t)tile * kTile;
            // the loaded tile into LDS
            float u[kOwn], zsl[kOwn];
            {
                const Mover<O> m(anew(l.tid), l.valid);
                float dt[kOwn], po[kOwn], slope[kOwn];
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    u[i] = to_f(ur[i]);
                    dt[i] = to_f(dr[i]) + par[min(max(m.channel(i), 0), kChannels - 1)].x;
                    po[i] = to_f(gr[i]);
                    slope[i] = 1.0f;
                    zsl[i] = to_f(zr[i]);
                }
                if (a.softplus) {
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) dt[i] = softplus_f<kFine<T>, true>(dt[i], &slope[i]);
                }
                if (gate) {
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) {
                        const float z = zsl[i], s = sigmoid_f<kFine<T>>(z);
                        zsl[i] = po[i] * s * fmaf(z, 1.0f - s, 1.0f);  // dz but for the ungated output
                        po[i] *= z * s;
                    }
                }
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    const bool in = m.step(i) < now;
                    dt[i] = in ? dt[i] : 0.0f;
                    po[i] = in ? po[i] : 0.0f;
                    if (ENDS) dtsum[i] += dt[i];
                    if (m.has(i, l.valid))
                        steps[m.step(i) * kStepRow + step_at(m.channel(i))] = make_float4(dt[i], dt[i] * u[i], po[i], slope[i]);
                }
                Stage<T, S>(a.B, a.C, N, anew(l.tid)).template store<!ENDS, true>(sb, sc, lds, now);
            }
            float h0[S];
            if (!ENDS) {
#pragma unroll
                for (int j = 0; j < S; ++j) h0[j] = hn[j];
            }
            __syncthreads();
            // the tile before this one, whole, flies while this one is run (the first
            // loads itself again where it is a whole one)
            if (tile > 0 || now == kTile) {
                const ScanGradArgs ga = arguments<ScanGradArgs>();
                const ScanArgs& a = ga.f;
                const View3& gv = a.z.data ? a.z : a.u;
                const int64_t back = tile > 0 ? kTile * (int64_t)sizeof(T) : 0;
                up -= back * a.u.sl, dp -= back * a.delta.sl, zp -= back * gv.sl, gp -= back * ga.dy.sl;
                Bp -= back * a.B.sl, Cp -= back * a.C.sl;
                const Mover<O> m(anew(l.tid), l.valid);
                m.template load<T>(ur, up, m.template offset<T>(a.u), a.u);
                m.template load<T>(dr, dp, m.template offset<T>(a.delta), a.delta);
                m.template load<T>(gr, gp, m.template offset<T>(ga.dy), ga.dy);
                m.template load<T>(zr, zp, m.template offset<T>(gv), gv);
                Stage<T, S>(a.B, a.C, N, anew(l.tid)).template load<!ENDS, true>(sb, sc, Bp, Cp);
                if (!ENDS) {
                    sv -= back ? wstep : 0;
                    load_states<S>(hn, sv);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            const float4* const bc = reinterpret_cast<const float4*>(lds) + p;
            const float4* const mine = steps + step_at(l.c);
            if constexpr (ENDS) {
                float4 dn = mine[(kTile - 1) * kStepRow], vn[S / 2];
#pragma unroll
                for (int k = 0; k < S / 2; ++k) vn[k] = bc[(kTile - 1) * (kRow / 4) + k * 8];
#pragma unroll
                for (int t = kTile - 1; t >= 0; --t) {
                    const float4 d = dn;
                    float4 vt[S / 2];
#pragma unroll
                    for (int k = 0; k < S / 2; ++k) vt[k] = vn[k];
                    if (t > 0) {
                        dn = mine[(t - 1) * kStepRow];
#pragma unroll
                        for (int k = 0; k < S / 2; ++k) vn[k] = bc[(t - 1) * (kRow / 4) + k * 8];
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = 0; k < S / 2; ++k) {
                        const float4 v = vt[k];
                        carry[2 * k] = fmaf(v.z, d.z, carry[2 * k]) * __builtin_amdgcn_exp2f(d.x * A2[2 * k]);
                        carry[2 * k + 1] =
                            fmaf(v.w, d.z, carry[2 * k + 1]) * __builtin_amdgcn_exp2f(d.x * A2[2 * k + 1]);
                    }
                }
                __syncthreads();
            } else {
#pragma unroll
                for (int k = 0; k < S / 2; ++k) {
                    // this pair of states through the tile and back
                    float dec[kTile][2], x[kTile + 1][2], share[4];
                    x[0][0] = h0[2 * k], x[0][1] = h0[2 * k + 1];
                    // LDS is read a step ahead of its use; without the barriers to scheduling
                    // the compiler puts the reads right before it, and waits every step
                    float2 dn = *reinterpret_cast<const float2*>(mine);
                    float4 vn = bc[k * 8];
#pragma unroll
                    for (int t = 0; t < kTile; ++t) {
                        const float2 d = dn;
                        const float4 v = vn;
                        if (t + 1 < kTile) {
                            dn = *reinterpret_cast<const float2*>(mine + (t + 1) * kStepRow);
                            vn = bc[(t + 1) * (kRow / 4) + k * 8];
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        dec[t][0] = __builtin_amdgcn_exp2f(d.x * A2[2 * k]);
                        dec[t][1] = __builtin_amdgcn_exp2f(d.x * A2[2 * k + 1]);
                        x[t + 1][0] = fmaf(dec[t][0], x[t][0], d.y * v.x);
                        x[t + 1][1] = fmaf(dec[t][1], x[t][1], d.y * v.y);
                        float y = fmaf(v.w, x[t + 1][1], v.z * x[t + 1][0]);
                        asm volatile("" : "+v"(y));  // the sum is done here, not where it is used
                        share[t & 3] = y;
                        if ((t & 3) == 3)
                            put_sums(ysum, t >> 2, quad_sums(share[0], share[1], share[2], share[3], odd, high), l.c, p,
                                     k > 0);
                    }
                    // on the way back B, C and the steps are read anew: kept from the way
                    // forth they would take eight registers per step
                    int again = 0;
                    asm volatile("" : "+v"(again));
                    const float4* const bc2 = bc + again;
                    const float4* const mine2 = mine + again;
                    float gshare[4], later = 0.0f;
                    float4 en = mine2[(kTile - 1) * kStepRow];
                    vn = bc2[(kTile - 1) * (kRow / 4) + k * 8];
#pragma unroll
                    for (int t = kTile - 1; t >= 0; --t) {
                        const float4 d = en, v = vn;
                        if (t > 0) {
                            en = mine2[(t - 1) * kStepRow];
                            vn = bc2[(t - 1) * (kRow / 4) + k * 8];
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        const float g0 = fmaf(v.z, d.z, carry[2 * k]), g1 = fmaf(v.w, d.z, carry[2 * k + 1]);
                        float gx = fmaf(g1, v.y, g0 * v.x);
                        carry[2 * k] = g0 * dec[t][0];
                        carry[2 * k + 1] = g1 * dec[t][1];
                        const float b0 = carry[2 * k] * x[t][0], b1 = carry[2 * k + 1] * x[t][1];
                        float dd = fmaf(b1, A2[2 * k + 1], b0 * A2[2 * k]);
                        dA[2 * k] = fmaf(b0, d.x, dA[2 * k]);
                        dA[2 * k + 1] = fmaf(b1, d.x, dA[2 * k + 1]);
                        const float s = channel_sums(g0 * d.y, g1 * d.y, d.z * x[t + 1][0], d.z * x[t + 1][1]);
                        // lane l holds number l >> 4 of {B, B, C, C}; lanes with bit 3 write the later step
                        if (t & 1) {
                            later = s;
                        } else {
                            red[(l.wave * kTile + t) * 32 + (bit3 ? 32 : 0) + (lane >> 5) * 16 + p * 2 +
                                ((lane >> 4) & 1)] = last_sums(s, later, bit3);
                        }
                        // these sums are done here too: their operands are a step's registers
                        asm volatile("" : "+v"(gx), "+v"(dd), "+v"(dA[2 * k]), "+v"(dA[2 * k + 1]));
                        share[t & 3] = dd;
                        gshare[t & 3] = gx;
                        if ((t & 3) == 0) {
                            put_sums(gsum, t >> 2, quad_sums(gshare[0], gshare[1], gshare[2], gshare[3], odd, high),
                                     l.c, p, k > 0);
                            put_sums(asum, t >> 2, quad_sums(share[0], share[1], share[2], share[3], odd, high), l.c, p,
                                     k > 0);
                        }
                    }
                    __syncthreads();
                    // the workgroup's sums of dB and dC: the eight waves' in order
                    constexpr int64_t kOut = S * 16;  // of a step and group
                    const ScanArgs a = arguments<ScanArgs>();
                    float* to = sp.part_bc + ((((int64_t)l.blk * a.Bsz + it.row) * a.q.L + t0) * a.G + l.g) * kOut;
#pragma unroll
                    for (int mm = 0; mm < 2; ++mm) {
                        const int e = l.tid + kScanThreads * mm, t = e >> 5;
                        float s = red[e];
#pragma unroll
                        for (int w = 1; w < 8; ++w) s += red[w * kTile * 32 + e];
                        if (t < now) to[(int64_t)t * a.G * kOut + k * 32 + (e & 31)] = s;
                    }
                    if (k + 1 < S / 2) __syncthreads();
                }
                // the tile's gradients
                const ScanGradArgs ga = arguments<ScanGradArgs>();
                const Mover<O> m(anew(l.tid), l.valid);
                float ys[kOwn], gs[kOwn], as[kOwn], o[kOwn];
                get_sums<O>(ys, ysum, m);
                get_sums<O>(gs, gsum, m);
                get_sums<O>(as, asum, m);
                float dt[kOwn], po[kOwn], slope[kOwn], Dv[kOwn];
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    Dv[i] = par[min(max(m.channel(i), 0), kChannels - 1)].y;
                    const float4 d = steps[m.step(i) * kStepRow + step_at(max(0, min(m.channel(i), l.valid - 1)))];
                    dt[i] = d.x, po[i] = d.z, slope[i] = d.w;
                    o[i] = fmaf(Dv[i], po[i], dt[i] * gs[i]);
                }
                m.template store<T>(o, dup, m.template offset<T>(ga.du), ga.du, l.valid, now);
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    o[i] = fmaf(u[i], gs[i], as[i] * kLn2) * slope[i];
                    dbsum[i] += m.step(i) < now ? o[i] : 0.0f;
                    dDsum[i] += m.step(i) < now ? po[i] * u[i] : 0.0f;
                }
                m.template store<T>(o, ddp, m.template offset<T>(ga.ddelta), ga.ddelta, l.valid, now);
                if (gate) {
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) o[i] = fmaf(Dv[i], u[i], ys[i]) * zsl[i];
                    m.template store<T>(o, dzp, m.template offset<T>(ga.dz), ga.dz, l.valid, now);
                }
                constexpr int64_t kBack = kTile * (int64_t)sizeof(T);
                dup -= kBack * ga.du.sl, ddp -= kBack * ga.ddelta.sl, dzp -= kBack * ga.dz.sl;
                __syncthreads();  // `steps` is read above and written next
            }
            now = kTile;
        }
    }

    // per channel, over the threads that moved its steps
    auto per_channel = [&](float (&v)[kOwn], float* out) {
        float* const part = reinterpret_cast<float*>(steps);
        constexpr int kParts = O == kRows ? 8 : kTile;
        __syncthreads();
#pragma unroll
        for (int i = 1; i < (O == kRows ? kOwn : 1); ++i) v[0] += v[i];
#pragma unroll
        for (int i = 0; i < (O == kRows ? 1 : kOwn); ++i)
            if (m.has(i, l.valid)) part[(O == kRows ? l.tid & 7 : m.t) * kChannels + m.channel(i)] = v[i];
        __syncthreads();
        if (l.tid < l.valid) {
            float s = 0.0f;
            for (int k = 0; k < kParts; ++k) s += part[k * kChannels + l.tid];
            out[l.first + l.tid] = s;
        }
    };
    if (ENDS) {
        per_channel(dtsum, sp.sums + item * a.H);
        if (l.live) store_states<S>(carry, sp.ends + item * wstep + wrow);
        return;
    }
    float* sums = sp.part + item * part_cols(a.H, 8 * S);
    per_channel(dDsum, sums + wstep);
    per_channel(dbsum, sums + wstep + a.H);
    if (!l.live) return;
    store_states<S>(dA, sums + wrow);
    if (work && it.c == 0 && ga.dx_in) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (p * S + j < N) ga.dx_in[((int64_t)it.s * a.H + l.h) * N + p * S + j] = carry[j];
    }
}

// dB and dC: the sums of a group's workgroups, four values a thread; steps
// outside every sequence stay as they were.  It reads per_group rows of 64 G S
// bytes per step and writes little, so HBM bounds it; sixteen loads a thread are in flight.
template <class T>
__device__ __forceinline__ void finish_bc(const ScanGradArgs& ga, const float* part, int per_group, int S, int64_t i) {
    const ScanArgs& a = ga.f;
    const int row = S * 4;
    const int64_t total = a.Bsz * a.q.L * a.G * row;
    if (i >= total) return;
    const int v = (int)(i & (row - 1)) * 4;
    const int64_t step = i / row, g = step % a.G, bl = step / a.G, b = bl / a.q.L;
    const int t = (int)(bl - b * a.q.L);
    int64_t r0;
    int beg, end, e0;
    if (a.q.offsets) {
        seq_bounds(a.q, 0, r0, beg, e0);
        seq_bounds(a.q, (int)a.q.S - 1, r0, e0, end);
    } else {
        seq_bounds(a.q, (int)b, r0, beg, end);
    }
    if (t < beg || t >= end) return;
    float s[4] = {};
    const float4* from = (const float4*)part + i;
    int k = 0;
    for (; k + 16 <= per_group; k += 16) {
        float4 x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = from[(k + j) * total];
#pragma unroll
        for (int j = 0; j < 16; ++j) s[0] += x[j].x, s[1] += x[j].y, s[2] += x[j].z, s[3] += x[j].w;
    }
    for (; k < per_group; ++k) {
        const float4 x = from[k * total];
        s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
    }
    const View4& o = v & 16 ? ga.dC : ga.dB;
    T* to = (T*)o.data + b * o.sb + g * o.sg + t * o.sl;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int w = v + j, n = ((w & 15) >> 1) * S + (w >> 5) * 2 + (w & 1);
        if (n < a.N) to[n * o.sn] = from_f<T>(s[j]);
    }
}

// dA, dD and ddelta_bias: the items' rows added in float64
constexpr int kSumCols = 32, kSumRows = 8;
__device__ __forceinline__ void finish_sums(const ScanGradArgs& ga, const GradSplit& sp, int64_t Np, int64_t block) {
    __shared__ double red[kSumRows][kSumCols];
    const ScanArgs& a = ga.f;
    const int c = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    const int64_t cols = part_cols(a.H, Np), col = block * kSumCols + c;
    double s = 0.0;
    if (col < cols)
        for (int64_t i = r; i < sp.items; i += kSumRows) s += (double)sp.part[i * cols + col];
    red[r][c] = s;
    __syncthreads();
    if (r != 0 || col >= cols) return;
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) s += red[i][c];
    if (col < a.H * Np) {
        const int64_t h = col / Np, n = col % Np;
        if (n < a.N) ga.dA[h * a.N + n] = (float)s;
    } else if (col < a.H * (Np + 1)) {
        if (ga.dD) ga.dD[col - a.H * Np] = (float)s;
    } else if (ga.ddelta_bias && col < a.H * (Np + 2)) {
        ga.ddelta_bias[col - a.H * (Np + 1)] = (float)s;
    }
}

template <class T>
__global__ __launch_bounds__(256) void grad_finish_kernel(ScanGradArgs ga, GradSplit sp, int S, unsigned sum_blocks) {
    if (blockIdx.x < sum_blocks)
        finish_sums(ga, sp, S * 8, blockIdx.x);
    else
        finish_bc<T>(ga, sp.part_bc, sp.per_group, S, (int64_t)(blockIdx.x - sum_blocks) * 256 + threadIdx.x);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
    GradSplit sp;
    int64_t items, Np;
    bool split;
    size_t ends, sums, bc, part;
};

Plan plan(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G) {
    Plan p;
    const int64_t Hg = H / G;
    p.sp.per_group = (int)((Hg + kChannels - 1) / kChannels);
    p.sp.blocks = (int)(G * p.sp.per_group);
    const int64_t Q = chunk_steps(q, p.sp.blocks, 3);
    p.sp.Q = (int)Q;
    p.split = Q < q.L;
    p.items = p.sp.items = item_count(q, Q);
    p.Np = padded_states(N);
    p.ends = p.split ? up256((size_t)p.items * H * p.Np * 4) : 0;
    p.sums = p.split ? up256((size_t)p.items * H * 4) : 0;
    p.bc = up256((size_t)p.sp.per_group * Bsz * q.L * G * p.Np * 2 * 4);
    p.part = up256((size_t)p.items * part_cols(H, p.Np) * 4);
    return p;
}

// workgroups of the last launch: dA, dD, ddelta_bias, then dB and dC
int64_t sum_blocks(int64_t H, int64_t Np) { return (part_cols(H, Np) + kSumCols - 1) / kSumCols; }
int64_t bc_blocks(int64_t Bsz, int64_t L, int64_t G, int64_t Np) { return (Bsz * L * G * (Np / 2) + 255) / 256; }

template <class T, int S, Order O>
hipError_t launch_as(const ScanGradArgs& g, const Plan& p, hipStream_t s) {
    const ScanArgs& a = g.f;
    const int64_t wgs = p.items * p.sp.blocks, sums = sum_blocks(a.H, p.Np);
    const int64_t finish = sums + bc_blocks(a.Bsz, a.q.L, a.G, p.Np);
    if (!grid_fits(wgs, kScanThreads) || !grid_fits(finish, 256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), lanes(kScanThreads);
    if (p.split) grad_kernel<T, S, O, true><<<grid, lanes, 0, s>>>(g, p.sp);
    grad_kernel<T, S, O, false><<<grid, lanes, 0, s>>>(g, p.sp);
    grad_finish_kernel<T><<<dim3((unsigned)finish), dim3(256), 0, s>>>(g, p.sp, S, (unsigned)sums);
    return hipGetLastError();
}

template <class T, int S>
hipError_t launch_in(const ScanGradArgs& g, const Plan& p, Order o, hipStream_t s) {
    return o == kRows ? launch_as<T, S, kRows>(g, p, s)
         : o == kTokens ? launch_as<T, S, kTokens>(g, p, s) : launch_as<T, S, kAny>(g, p, s);
}

template <class T>
hipError_t launch_of(const ScanGradArgs& g, const Plan& p, Order o, hipStream_t s) {
    if (g.f.N <= 16) return launch_in<T, 2>(g, p, o, s);
    if (g.f.N <= 32) return launch_in<T, 4>(g, p, o, s);
    return launch_in<T, 8>(g, p, o, s);
}

}  // namespace

size_t scan_grad_workspace_bytes(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, Bsz, H, N, G);
    return p.ends + p.sums + p.bc + p.part;
}

bool scan_grad_fits(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, Bsz, H, N, G);
    return grid_fits(p.items * p.sp.blocks, kScanThreads) &&
           grid_fits(sum_blocks(H, p.Np) + bc_blocks(Bsz, q.L, G, p.Np), 256);
}

hipError_t launch_scan_backward(int dtype, const ScanGradArgs& g, void* ws, hipStream_t s) {
    const ScanArgs& a = g.f;
    Plan p = plan(a.q, a.Bsz, a.H, a.N, a.G);
    char* at = (char*)ws;
    auto take = [&](size_t bytes) {
        float* r = (float*)at;
        at += bytes;
        return r;
    };
    p.sp.ends = take(p.ends);
    p.sp.sums = take(p.sums);
    p.sp.part_bc = take(p.bc);
    p.sp.part = take(p.part);
    const View3* views[] = {&a.u, &a.delta, &a.z, &g.dy, &g.du, &g.ddelta, &g.dz};
    const Order o = order_of(views, 7, a.H / a.G);
    if (dtype == SSM_F32) return launch_of<float>(g, p, o, s);
    if (dtype == SSM_BF16) return launch_of<bf16>(g, p, o, s);
    return launch_of<f16>(g, p, o, s);
}

}  // namespace ssm

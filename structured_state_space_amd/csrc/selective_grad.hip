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
// Work split as in the forward scan: eight lanes per channel, 8 channels per
// wave, 64 per workgroup.  The workgroup takes the tiles of 32 steps from the
// last to the first, recomputes a tile's states from the one that the forward
// pass saved at its first step (states and decays stay in registers, for one
// pair of a lane's states at a time) and walks back through it.
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
#include "selective.hpp"

namespace ssm {

namespace {

// sums over the 8 channels of a wave (lane bits 3..5) of four values per lane:
// lane l gets the sum of its lane position's value number l >> 4
__device__ __forceinline__ float channel_sums(float v0, float v1, float v2, float v3) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v0), __float_as_uint(v2), false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v1), __float_as_uint(v3), false, false);
    const float x = __uint_as_float(a[0]) + __uint_as_float(a[1]);  // v0 below lane 32, v2 above
    const float y = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    const float s = __uint_as_float(c[0]) + __uint_as_float(c[1]);
    return s + dpp<0x128>(s);  // row_ror:8
}

struct GradSplit {
    int Q, blocks, per_group;
    int64_t items;  // work items launched
    float* ends;    // [items, H, Np]: gradient a chunk hands to the chunk before it, from a zero end
    float* sums;    // [items, H]: sum of dt over a chunk
    float* part_bc; // [per_group, Bsz, L, G, S/2, 2, 16]: a workgroup's dB and dC by pairs of lane states
    float* part_a;  // [items, H, Np]
    float* part_d;  // [items, 2, H]: dD, ddelta_bias
};

template <class T, int S, bool ROWS, bool ENDS>
__global__ __launch_bounds__(kScanThreads, 2) void grad_kernel(ScanGradArgs ga, GradSplit sp) {
    const ScanArgs& a = ga.f;
    using St = Stage<T, S>;
    constexpr int kRow = St::kRow;
    __shared__ __attribute__((aligned(16))) float lds[2][kTile * kRow];
    __shared__ float red[ENDS ? 1 : 8 * kTile * 32];

    const int cb = blockIdx.x % sp.blocks;
    const int64_t item = blockIdx.x / sp.blocks;
    Item it;
    const bool there = find_item(a.q, item, sp.Q, it);
    const Place l = place_of(cb, sp.per_group, a.H, a.G);
    const int p = l.p, N = (int)a.N, lane = l.tid & 63;
    const bool odd = p & 1, high = p & 2, upper = p & 4;
    const int64_t wrow = (int64_t)l.h * (8 * S) + p * S, wstep = a.H * (8 * S);

    float A2[S], carry[S], dA[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        A2[j] = p * S + j < N ? a.A[(int64_t)l.h * N + p * S + j] * kLog2e : 0.0f;
        carry[j] = dA[j] = 0.0f;
    }
    float dDsum = 0.0f, dbsum = 0.0f, dtsum = 0.0f;

    const int chunks = there ? chunks_of(it.end - it.beg, sp.Q) : 0;
    const int beg = there ? it.beg + it.c * sp.Q : 0;
    const int end = there ? (int)min((int64_t)it.end, (int64_t)beg + sp.Q) : 0;
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
#pragma unroll
                for (int j = 0; j < S; ++j) carry[j] = fmaf(__builtin_amdgcn_exp2f(s * A2[j]), carry[j], e[j]);
            }
        }
    }

    if (work && beg < end) {
        const float bias = a.delta_bias ? a.delta_bias[l.h] : 0.0f;
        const float Dv = a.D ? a.D[l.h] : 0.0f;
        const bool gate = a.z.data;
        const int last = beg + (end - 1 - beg) / kTile * kTile;  // the last tile's first step
        constexpr uint32_t kE = sizeof(T);
        const uint32_t q0 = step_of<ROWS>(p, 0);
        auto base = [&](const View3& v) {
            return (char*)v.data + (it.row * v.sb + l.w0 * v.sh + last * v.sl) * (int64_t)kE;
        };
        auto offset = [&](const View3& v) { return (l.dh * (uint32_t)v.sh + q0 * (uint32_t)v.sl) * kE; };
        auto step4 = [&](const View3& v) { return (uint32_t)v.sl * 4 * kE; };
        const View3& gv = gate ? a.z : a.u;  // without a gate u once more, unused
        const char *up = base(a.u), *dp = base(a.delta), *zp = base(gv), *gp = base(ga.dy);
        char *dup = base(ga.du), *ddp = base(ga.ddelta), *dzp = base(ga.dz);
        const uint32_t uo = offset(a.u), dof = offset(a.delta), zo = offset(gv), go = offset(ga.dy);
        const uint32_t us = step4(a.u), ds = step4(a.delta), zs = step4(gv), gs = step4(ga.dy);
        const char* Bp = (const char*)a.B.data + (it.row * a.B.sb + l.g * a.B.sg + last * a.B.sl) * (int64_t)kE;
        const char* Cp = (const char*)a.C.data + (it.row * a.C.sb + l.g * a.C.sg + last * a.C.sl) * (int64_t)kE;
        const uint32_t bs = (uint32_t)a.B.sl * 4 * kE, cs = (uint32_t)a.C.sl * 4 * kE;
        St stage;
        stage.init(a.B, a.C, N, l.tid);
        const float* sv = ENDS ? nullptr : ga.saved + (saved_row(a.q, it) + (last - it.beg) / kTile) * wstep + wrow;

        T ur[kOwn], dr[kOwn], zr[kOwn], gr[kOwn];
        float hn[S];
        // the last tile may be a part of one
        int now = end - last;
        load_part<T, ROWS>(ur, up, uo, us, now, p);
        load_part<T, ROWS>(dr, dp, dof, ds, now, p);
        load_part<T, ROWS>(gr, gp, go, gs, now, p);
        load_part<T, ROWS>(zr, zp, zo, zs, now, p);
        stage.template load_part<!ENDS, true>(Bp, Cp, now);
        stage.template store<!ENDS, true>(lds[0]);
        if (!ENDS) load_states<S>(hn, sv);
        __syncthreads();
        int buf = 0;
        for (int t0 = last; t0 >= beg; t0 -= kTile) {
            float u[kOwn], slope[kOwn], zsl[kOwn];
            float dt[2][kOwn], dx[2][kOwn], pv[2][kOwn];
            float own[kOwn], po[kOwn];  // dt, and dy behind the gate
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                u[i] = to_f(ur[i]);
                own[i] = to_f(dr[i]) + bias;
                po[i] = to_f(gr[i]);
                slope[i] = 1.0f;
                zsl[i] = to_f(zr[i]);
            }
            if (a.softplus) {
#pragma unroll
                for (int i = 0; i < kOwn; ++i) own[i] = softplus_f<kFine<T>, true>(own[i], &slope[i]);
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
                const bool in = step_of<ROWS>(p, i) < now;
                own[i] = in ? own[i] : 0.0f;
                po[i] = in && l.live ? po[i] : 0.0f;
                if (ENDS) dtsum += own[i];
                both_halves(own[i], dt[0][i], dt[1][i]);
                both_halves(po[i], pv[0][i], pv[1][i]);
                if (!ENDS) both_halves(own[i] * u[i], dx[0][i], dx[1][i]);
            }
            float h0[S];
            if (!ENDS) {
#pragma unroll
                for (int j = 0; j < S; ++j) h0[j] = hn[j];
            }
            // the tile before this one, whole, flies while this one is computed (the
            // first loads a whole tile's worth of itself again where it is one)
            const uint32_t back = t0 > beg ? kTile / 4 : 0;
            if (t0 > beg || now == kTile) {
                up -= (uint64_t)us * back, dp -= (uint64_t)ds * back, zp -= (uint64_t)zs * back;
                gp -= (uint64_t)gs * back, Bp -= (uint64_t)bs * back, Cp -= (uint64_t)cs * back;
                load_own<T, ROWS>(ur, up, uo, us);
                load_own<T, ROWS>(dr, dp, dof, ds);
                load_own<T, ROWS>(gr, gp, go, gs);
                load_own<T, ROWS>(zr, zp, zo, zs);
                stage.template load<!ENDS, true>(Bp, Cp);
                if (!ENDS) {
                    sv -= back ? wstep : 0;
                    load_states<S>(hn, sv);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            const float4* const bc = reinterpret_cast<const float4*>(&lds[0][0]);
            int bq = buf * (kTile * kRow / 4) + p;  // the lane's B and C in it
            if constexpr (ENDS) {
#pragma unroll
                for (int t = kTile - 1; t >= 0; --t) {
                    const float dtv = quad_bcast(dt[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
                    const float pt = quad_bcast(pv[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
#pragma unroll
                    for (int k = 0; k < S / 2; ++k) {
                        const float4 v = bc[bq + t * (kRow / 4) + k * 8];
                        carry[2 * k] = fmaf(v.z, pt, carry[2 * k]) * __builtin_amdgcn_exp2f(dtv * A2[2 * k]);
                        carry[2 * k + 1] =
                            fmaf(v.w, pt, carry[2 * k + 1]) * __builtin_amdgcn_exp2f(dtv * A2[2 * k + 1]);
                    }
                }
            } else {
                float ys[kOwn] = {}, gxs[kOwn] = {}, dds[kOwn] = {};
#pragma unroll
                for (int k = 0; k < S / 2; ++k) {
                    // this pair of states through the tile and back
                    float dec[kTile][2], x[kTile + 1][2];
                    float sums[2][kOwn], share[16];
                    auto collect = [&](int t) {  // the lanes' shares of the steps up to t (forth) or from t on (back)
                        if (!ROWS)
                            sums[t >> 4][(t >> 2) & 3] = quad_sums(share[0], share[1], share[2], share[3], odd, high);
                        if (ROWS) {
#pragma unroll
                            for (int i = 0; i < kOwn; ++i)
                                sums[t >> 4][i] =
                                    quad_sums(share[i], share[4 + i], share[8 + i], share[12 + i], odd, high);
                        }
                    };
                    x[0][0] = h0[2 * k], x[0][1] = h0[2 * k + 1];
#pragma unroll
                    for (int t = 0; t < kTile; ++t) {
                        const float dtv = quad_bcast(dt[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
                        const float dxv = quad_bcast(dx[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
                        const float4 v = bc[bq + t * (kRow / 4) + k * 8];
                        dec[t][0] = __builtin_amdgcn_exp2f(dtv * A2[2 * k]);
                        dec[t][1] = __builtin_amdgcn_exp2f(dtv * A2[2 * k + 1]);
                        x[t + 1][0] = fmaf(dec[t][0], x[t][0], dxv * v.x);
                        x[t + 1][1] = fmaf(dec[t][1], x[t][1], dxv * v.y);
                        float y = fmaf(v.w, x[t + 1][1], v.z * x[t + 1][0]);
                        asm volatile("" : "+v"(y));  // the sum is done here, not where it is used
                        share[ROWS ? t & 15 : t & 3] = y;
                        if (t % (ROWS ? 16 : 4) == (ROWS ? 15 : 3)) collect(t);
                    }
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) ys[i] += half_sums(sums[0][i], sums[1][i], upper);
                    float dsum[2][kOwn], dshare[16];
                    // on the way back B, C and the passed-on values are read anew: kept
                    // from the way forth they would take six registers per step
                    asm volatile("" : "+v"(bq));
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
                        asm volatile("" : "+v"(dt[0][i]), "+v"(dt[1][i]), "+v"(dx[0][i]), "+v"(dx[1][i]));
#pragma unroll
                    for (int t = kTile - 1; t >= 0; --t) {
                        const float dtv = quad_bcast(dt[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
                        const float dxv = quad_bcast(dx[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
                        const float pt = quad_bcast(pv[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
                        const float4 v = bc[bq + t * (kRow / 4) + k * 8];
                        const float g0 = fmaf(v.z, pt, carry[2 * k]), g1 = fmaf(v.w, pt, carry[2 * k + 1]);
                        float gx = fmaf(g1, v.y, g0 * v.x);
                        carry[2 * k] = g0 * dec[t][0];
                        carry[2 * k + 1] = g1 * dec[t][1];
                        const float b0 = carry[2 * k] * x[t][0], b1 = carry[2 * k + 1] * x[t][1];
                        float dd = fmaf(b1, A2[2 * k + 1], b0 * A2[2 * k]);
                        dA[2 * k] = fmaf(b0, dtv, dA[2 * k]);
                        dA[2 * k + 1] = fmaf(b1, dtv, dA[2 * k + 1]);
                        const float s = channel_sums(g0 * dxv, g1 * dxv, pt * x[t + 1][0], pt * x[t + 1][1]);
                        // [wave][t][B or C][n]: lane l holds number l >> 4 of {B, B, C, C}
                        if ((lane & 8) == 0)
                            red[(l.wave * kTile + t) * 32 + (lane >> 5) * 16 + p * 2 + ((lane >> 4) & 1)] = s;
                        // these sums are done here too: their operands are a step's registers
                        asm volatile("" : "+v"(gx), "+v"(dd), "+v"(dA[2 * k]), "+v"(dA[2 * k + 1]));
                        share[ROWS ? t & 15 : t & 3] = gx;
                        dshare[ROWS ? t & 15 : t & 3] = dd;
                        if (t % (ROWS ? 16 : 4) == 0) {
                            collect(t);
#pragma unroll
                            for (int i = 0; i < (ROWS ? kOwn : 1); ++i)
                                dsum[t >> 4][ROWS ? i : (t >> 2) & 3] =
                                    ROWS ? quad_sums(dshare[i], dshare[(4 + i) & 15], dshare[(8 + i) & 15],
                                                     dshare[(12 + i) & 15], odd, high)
                                         : quad_sums(dshare[0], dshare[1], dshare[2], dshare[3], odd, high);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) {
                        gxs[i] += half_sums(sums[0][i], sums[1][i], upper);
                        dds[i] += half_sums(dsum[0][i], dsum[1][i], upper);
                    }
                    __syncthreads();
                    // the workgroup's sums of dB and dC: the eight waves' in order
                    constexpr int64_t kOut = S * 16;  // of a step and group
                    float* to = sp.part_bc + ((((int64_t)l.blk * a.Bsz + it.row) * a.q.L + t0) * a.G + l.g) * kOut;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int e = l.tid + kScanThreads * m, t = e >> 5;
                        if (t < now) {
                            float s = red[e];
#pragma unroll
                            for (int w = 1; w < 8; ++w) s += red[w * kTile * 32 + e];
                            to[(int64_t)t * a.G * kOut + k * 32 + (e & 31)] = s;
                        }
                    }
                    if (k + 1 < S / 2) __syncthreads();
                }
                float o[kOwn];
#pragma unroll
                for (int i = 0; i < kOwn; ++i)
                    o[i] = fmaf(Dv, upper ? pv[1][i] : pv[0][i], (upper ? dt[1][i] : dt[0][i]) * gxs[i]);
                if (l.live) store_own<T, ROWS>(o, dup, offset(ga.du), step4(ga.du), now, p);
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    o[i] = fmaf(u[i], gxs[i], dds[i] * kLn2) * slope[i];
                    if (step_of<ROWS>(p, i) < now) {
                        dbsum += o[i];
                        dDsum = fmaf(upper ? pv[1][i] : pv[0][i], u[i], dDsum);
                    }
                }
                if (l.live) store_own<T, ROWS>(o, ddp, offset(ga.ddelta), step4(ga.ddelta), now, p);
                if (gate) {
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) o[i] = fmaf(Dv, u[i], ys[i]) * zsl[i];
                    if (l.live) store_own<T, ROWS>(o, dzp, offset(ga.dz), step4(ga.dz), now, p);
                }
                dup -= (uint64_t)step4(ga.du) * (kTile / 4), ddp -= (uint64_t)step4(ga.ddelta) * (kTile / 4);
                dzp -= (uint64_t)step4(ga.dz) * (kTile / 4);
            }
            now = kTile;
            buf ^= 1;
            stage.template store<!ENDS, true>(lds[buf]);
            __syncthreads();
        }
    }

    if (ENDS) {
        dtsum = lane_sum(dtsum);
        if (l.live) {
            store_states<S>(carry, sp.ends + item * wstep + wrow);
            if (p == 0) sp.sums[item * a.H + l.h] = dtsum;
        }
        return;
    }
    dDsum = lane_sum(dDsum);
    dbsum = lane_sum(dbsum);
    if (!l.live) return;
    store_states<S>(dA, sp.part_a + item * wstep + wrow);
    if (p == 0) {
        sp.part_d[(item * 2) * a.H + l.h] = dDsum;
        sp.part_d[(item * 2 + 1) * a.H + l.h] = dbsum;
    }
    if (work && it.c == 0 && ga.dx_in) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (p * S + j < N) ga.dx_in[((int64_t)it.s * a.H + l.h) * N + p * S + j] = carry[j];
    }
}

// dB and dC from the workgroups' sums; steps outside every sequence stay as they were
template <class T>
__global__ __launch_bounds__(256) void grad_bc_kernel(ScanGradArgs ga, const float* part, int per_group, int S) {
    const ScanArgs& a = ga.f;
    const int64_t row = (int64_t)S * 16, total = a.Bsz * a.q.L * a.G * row;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int v = (int)(i % row);
    const int g = (int)(i / row % a.G);
    const int64_t bl = i / (row * a.G);
    const int64_t b = bl / a.q.L;
    const int t = (int)(bl % a.q.L), n = ((v & 15) >> 1) * S + (v >> 5) * 2 + (v & 1);
    if (n >= a.N) return;
    int64_t r0;
    int beg, end, e0;
    if (a.q.offsets) {
        seq_bounds(a.q, 0, r0, beg, e0);
        seq_bounds(a.q, (int)a.q.S - 1, r0, e0, end);
    } else {
        seq_bounds(a.q, (int)b, r0, beg, end);
    }
    if (t < beg || t >= end) return;
    float s = part[i];
    for (int k = 1; k < per_group; ++k) s += part[(int64_t)k * total + i];
    const View4& o = v & 16 ? ga.dC : ga.dB;
    ((T*)o.data)[b * o.sb + g * o.sg + n * o.sn + t * o.sl] = from_f<T>(s);
}

// dA, dD and ddelta_bias: the workgroups' rows added in float64
constexpr int kSumCols = 32, kSumRows = 8;
__global__ __launch_bounds__(256) void grad_sum_kernel(const float* part, int64_t rows, int64_t cols, int64_t stride,
                                                       int width, int kept, float* out) {
    // columns are [cols / width] runs of `width`, of which the first `kept` go to `out`
    __shared__ double red[kSumRows][kSumCols];
    const int c = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    const int64_t col = (int64_t)blockIdx.x * kSumCols + c;
    double s = 0.0;
    if (col < cols)
        for (int64_t i = r; i < rows; i += kSumRows) s += (double)part[i * stride + col];
    red[r][c] = s;
    __syncthreads();
    if (r == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) s += red[i][c];
        const int64_t h = col / width, n = col % width;
        if (n < kept) out[h * kept + n] = (float)s;
    }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
    GradSplit sp;
    int64_t items, Np;
    bool split;
    size_t ends, sums, bc, pa, pd;
};

Plan plan(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G) {
    constexpr int64_t kFew = 256, kMany = 512;
    Plan p;
    const int64_t Hg = H / G;
    p.sp.per_group = (int)((Hg + kChannels - 1) / kChannels);
    p.sp.blocks = (int)(G * p.sp.per_group);
    const int64_t rows = q.offsets ? 1 : q.S;
    int64_t Q = q.L;
    if (q.offsets || rows * p.sp.blocks < kFew) {
        const int64_t share = (q.L * rows * p.sp.blocks + kMany - 1) / kMany;
        Q = share < q.L ? share : q.L;
        if (Q < 2 * kTile) Q = 2 * kTile;
    }
    Q = (Q + kTile - 1) / kTile * kTile;
    if (Q > ((int64_t)1 << 30)) Q = (int64_t)1 << 30;
    p.sp.Q = (int)Q;
    p.split = Q < q.L;
    p.items = p.sp.items = item_count(q, Q);
    p.Np = padded_states(N);
    p.ends = p.split ? up256((size_t)p.items * H * p.Np * 4) : 0;
    p.sums = p.split ? up256((size_t)p.items * H * 4) : 0;
    p.bc = up256((size_t)p.sp.per_group * Bsz * q.L * G * p.Np * 2 * 4);
    p.pa = up256((size_t)p.items * H * p.Np * 4);
    p.pd = up256((size_t)p.items * H * 2 * 4);
    return p;
}

template <class T, int S, bool ROWS>
hipError_t launch_as(const ScanGradArgs& g, const Plan& p, hipStream_t s) {
    const ScanArgs& a = g.f;
    const int64_t wgs = p.items * p.sp.blocks;
    const int64_t bc = (a.Bsz * a.q.L * a.G * S * 16 + 255) / 256;
    if (wgs >= ((int64_t)1 << 31) || bc >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), wg(256), lanes(kScanThreads);
    if (p.split) grad_kernel<T, S, ROWS, true><<<grid, lanes, 0, s>>>(g, p.sp);
    grad_kernel<T, S, ROWS, false><<<grid, lanes, 0, s>>>(g, p.sp);
    grad_bc_kernel<T><<<dim3((unsigned)bc), wg, 0, s>>>(g, p.sp.part_bc, p.sp.per_group, S);
    auto sum = [&](const float* part, int64_t cols, int64_t stride, int width, int kept, float* out) {
        grad_sum_kernel<<<dim3((unsigned)((cols + kSumCols - 1) / kSumCols)), wg, 0, s>>>(part, p.items, cols, stride,
                                                                                        width, kept, out);
    };
    sum(p.sp.part_a, a.H * p.Np, a.H * p.Np, (int)p.Np, (int)a.N, g.dA);
    if (g.dD) sum(p.sp.part_d, a.H, 2 * a.H, 1, 1, g.dD);
    if (g.ddelta_bias) sum(p.sp.part_d + a.H, a.H, 2 * a.H, 1, 1, g.ddelta_bias);
    return hipGetLastError();
}

template <class T>
hipError_t launch_of(const ScanGradArgs& g, const Plan& p, bool rows, hipStream_t s) {
    const int64_t N = g.f.N;
    if (N <= 16) return rows ? launch_as<T, 2, true>(g, p, s) : launch_as<T, 2, false>(g, p, s);
    if (N <= 32) return rows ? launch_as<T, 4, true>(g, p, s) : launch_as<T, 4, false>(g, p, s);
    return rows ? launch_as<T, 8, true>(g, p, s) : launch_as<T, 8, false>(g, p, s);
}

}  // namespace

size_t scan_grad_workspace_bytes(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, Bsz, H, N, G);
    return p.ends + p.sums + p.bc + p.pa + p.pd;
}

bool scan_grad_fits(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, Bsz, H, N, G);
    return p.items * p.sp.blocks < ((int64_t)1 << 31) && Bsz * q.L * G * p.Np * 2 / 256 < ((int64_t)1 << 31) - 1;
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
    p.sp.part_a = take(p.pa);
    p.sp.part_d = take(p.pd);
    const View3* views[] = {&a.u, &a.delta, &a.z, &g.dy, &g.du, &g.ddelta, &g.dz};
    bool rows = true;
    for (const View3* v : views) rows = rows && (!v->data || v->sl == 1);
    if (dtype == SSM_F32) return launch_of<float>(g, p, rows, s);
    if (dtype == SSM_BF16) return launch_of<bf16>(g, p, rows, s);
    return launch_of<f16>(g, p, rows, s);
}

}  // namespace ssm

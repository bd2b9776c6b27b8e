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
// Work split as in the forward scan: a quad of lanes per channel, 16 channels
// per wave, 64 per workgroup.  A tile is the kSaveSteps steps between two
// states that the forward pass saved: the workgroup takes the tiles from the
// last to the first, recomputes a tile's states from its saved one (they and
// the decays stay in registers) and walks back through it.
//
// dB and dC are sums over all channels of a group: over a wave's 16 channels by
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

constexpr int kT = kSaveSteps;  // steps of a tile: 16
constexpr int kOwn = kT / 4;    // of them a lane's own
constexpr int kChannels = 64;

template <bool ROWS>
constexpr int owner(int t) { return ROWS ? t / kOwn : t & 3; }
template <bool ROWS>
constexpr int reg(int t) { return ROWS ? t % kOwn : t >> 2; }
template <bool ROWS>
__device__ __forceinline__ int step_of(int q, int r) { return ROWS ? q * kOwn + r : r * 4 + q; }

template <class T, bool ROWS>
__device__ __forceinline__ void load4(T (&r)[kOwn], const T* base, uint32_t off, int64_t sl, int nt, int q) {
    if (nt == kT) {
        if constexpr (ROWS) {
            const Vec4<T> v = *reinterpret_cast<const Vec4<T>*>(base + off);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) r[i] = v.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < kOwn; ++i, base += 4 * sl) r[i] = base[off];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kOwn; ++i, base += ROWS ? 1 : 4 * sl)
            r[i] = step_of<ROWS>(q, i) < nt ? base[off] : from_f<T>(0.0f);
    }
}
template <class T, bool ROWS>
__device__ __forceinline__ void store4(const float (&v)[kOwn], T* base, uint32_t off, int64_t sl, int nt, int q) {
    if (nt == kT) {
        if constexpr (ROWS) {
            Vec4<T> w;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) w.v[i] = from_f<T>(v[i]);
            *reinterpret_cast<Vec4<T>*>(base + off) = w;
        } else {
#pragma unroll
            for (int i = 0; i < kOwn; ++i, base += 4 * sl) base[off] = from_f<T>(v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kOwn; ++i, base += ROWS ? 1 : 4 * sl)
            if (step_of<ROWS>(q, i) < nt) base[off] = from_f<T>(v[i]);
    }
}

// softplus and its slope e / (1 + e)
__device__ __forceinline__ float softplus_slope_f(float v, float& slope) {
    const float e = exp_f(fminf(v, 20.0f));
    const float w = 1.0f + e;
    const float c = e < 1.0f ? e - (w - 1.0f) : 0.0f;
    const float r = fmaf(__builtin_amdgcn_logf(w), kLn2, c);
    slope = v > 20.0f ? 1.0f : (v == v ? e * __builtin_amdgcn_rcpf(w) : v);
    return v > 20.0f ? v : (v == v ? r : v);
}

// sums over the 16 channels of a wave (lane bits 2..5) of eight values per
// lane; lane l of a row of 16 gets, of its quad position's values, number
// 4 (l >> 5) + 2 (l >> 4 & 1) in s0 and the next in s1
__device__ __forceinline__ void channel_sums(float (&v)[8], float& s0, float& s1) {
    float w[4], x[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 4]), false, false);
        w[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[i]), __float_as_uint(w[i + 2]), false, false);
        x[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        x[i] += dpp<0x124>(x[i]);  // row_ror:4
        x[i] += dpp<0x128>(x[i]);  // row_ror:8
    }
    s0 = x[0], s1 = x[1];
}

struct GradSplit {
    int Q, blocks, per_group;
    int64_t items;  // work items launched
    float* ends;    // [items, H, Np]: gradient a chunk hands to the chunk before it, from a zero end
    float* sums;    // [items, H]: sum of dt over a chunk
    float* part_bc; // [per_group, Bsz, L, G, NB, 2, 16]: a workgroup's dB and dC
    float* part_a;  // [items, H, Np]
    float* part_d;  // [items, 2, H]: dD, ddelta_bias
};

template <class T, int NB, bool ROWS, bool ENDS>
__global__ __launch_bounds__(256, NB == 1 ? 2 : 1) void grad_kernel(ScanGradArgs ga, GradSplit sp) {
    const ScanArgs& a = ga.f;
    constexpr int kPad = NB * 32 + 4;
    __shared__ __attribute__((aligned(16))) float lds[2][kT * kPad];
    __shared__ __attribute__((aligned(16))) float red[ENDS ? 1 : 4 * kT * NB * 32];

    const int cb = blockIdx.x % sp.blocks;
    const int64_t item = blockIdx.x / sp.blocks;
    Item it;
    const bool there = find_item(a.q, item, sp.Q, it);
    const int tid = threadIdx.x, lane = tid & 63, q = lane & 3, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool odd = q & 1, high = q & 2;
    const int Hg = (int)(a.H / a.G), N = (int)a.N, Np = NB * 16;
    const int g = cb / sp.per_group, blk = cb % sp.per_group;
    const int c0 = blk * kChannels + wave * 16;
    const int lc = lane >> 2;
    const bool live = c0 + lc < Hg;
    const int w0 = g * Hg + min(c0, Hg - 1);
    const int h0 = g * Hg + min(c0 + lc, Hg - 1);
    const uint32_t dh = (uint32_t)(h0 - w0);
    const int64_t wrow = (int64_t)h0 * Np + q * 4, wstep = a.H * Np;

    float A2[NB][4], carry[NB][4], dA[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = nb * 16 + q * 4 + j;
            A2[nb][j] = n < N ? a.A[(int64_t)h0 * N + n] * kLog2e : 0.0f;
            carry[nb][j] = dA[nb][j] = 0.0f;
        }
    float dDsum = 0.0f, dbsum = 0.0f, dtsum = 0.0f;

    const int chunks = there ? chunks_of(it.end - it.beg, sp.Q) : 0;
    const int beg = there ? it.beg + it.c * sp.Q : 0;
    const int end = there ? (int)min((int64_t)it.end, (int64_t)beg + sp.Q) : 0;
    const bool work = there && it.c < chunks && (!ENDS || it.c > 0);
    if (ENDS && !work) return;
    if (work) {
        // the gradient that the steps behind this chunk hand to its last state
        if (it.c + 1 == chunks) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = nb * 16 + q * 4 + j;
                    if (ga.dx_out && live && n < N) carry[nb][j] = ga.dx_out[((int64_t)it.s * a.H + h0) * N + n];
                }
        } else if (!ENDS) {
            // (descending offsets may name more items than there are)
            const int64_t from = min(item + (chunks - 1 - it.c), sp.items - 1);
            for (int64_t i = from; i > item; --i) {
                const float s = sp.sums[i * a.H + h0];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float4 v = *reinterpret_cast<const float4*>(sp.ends + i * wstep + wrow + nb * 16);
                    const float e[4] = {live ? v.x : 0.0f, live ? v.y : 0.0f, live ? v.z : 0.0f, live ? v.w : 0.0f};
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // the last chunk's holds dx_out's part already
                        carry[nb][j] = i == from
                                           ? e[j]
                                           : fmaf(__builtin_amdgcn_exp2f(s * A2[nb][j]), carry[nb][j], e[j]);
                }
            }
        }
    }

    if (work && beg < end) {
        const float bias = a.delta_bias ? a.delta_bias[h0] : 0.0f;
        const float Dv = a.D ? a.D[h0] : 0.0f;
        const bool gate = a.z.data;
        const int last = beg + (end - 1 - beg) / kT * kT;  // the last tile's first step
        const T* up = (const T*)a.u.data + it.row * a.u.sb + w0 * a.u.sh + last * a.u.sl;
        const T* dp = (const T*)a.delta.data + it.row * a.delta.sb + w0 * a.delta.sh + last * a.delta.sl;
        const T* zp = (const T*)a.z.data + it.row * a.z.sb + w0 * a.z.sh + last * a.z.sl;
        const T* gp = (const T*)ga.dy.data + it.row * ga.dy.sb + w0 * ga.dy.sh + last * ga.dy.sl;
        T* dup = (T*)ga.du.data + it.row * ga.du.sb + w0 * ga.du.sh + last * ga.du.sl;
        T* ddp = (T*)ga.ddelta.data + it.row * ga.ddelta.sb + w0 * ga.ddelta.sh + last * ga.ddelta.sl;
        T* dzp = (T*)ga.dz.data + it.row * ga.dz.sb + w0 * ga.dz.sh + last * ga.dz.sl;
        const uint32_t q0 = ROWS ? q * kOwn : q;
        auto offset = [&](const View3& v) { return dh * (uint32_t)v.sh + q0 * (uint32_t)v.sl; };
        const T* Bp = (const T*)a.B.data + it.row * a.B.sb + g * a.B.sg + last * a.B.sl;
        const T* Cp = (const T*)a.C.data + it.row * a.C.sb + g * a.C.sg + last * a.C.sl;
        const bool by_time = a.B.sl == 1;
        T sb[NB], sc[NB];
        auto stage_pos = [&](int k, int& t, int& n) {
            const int e = tid + 256 * k;
            t = by_time ? e % kT : e / (NB * 16);
            n = by_time ? e / kT : e % (NB * 16);
        };
        auto stage_load = [&](int nt) {
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                int t, n;
                stage_pos(k, t, n);
                const bool in = t < nt && n < N;
                if (!ENDS)
                    sb[k] = in ? Bp[(uint32_t)n * (uint32_t)a.B.sn + (uint32_t)t * (uint32_t)a.B.sl] : from_f<T>(0.0f);
                sc[k] = in ? Cp[(uint32_t)n * (uint32_t)a.C.sn + (uint32_t)t * (uint32_t)a.C.sl] : from_f<T>(0.0f);
            }
        };
        auto stage_store = [&](float* to) {
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                int t, n;
                stage_pos(k, t, n);
                float* at = to + t * kPad + (n >> 2) * 8 + (n & 3);
                if (!ENDS) at[0] = to_f(sb[k]);
                at[4] = to_f(sc[k]);
            }
        };
        const float* sv = nullptr;
        float4 hn[NB];
        if (!ENDS) sv = ga.saved + (saved_row(a.q, it) + (last - it.beg) / kT) * wstep + wrow;

        T ur[kOwn], dr[kOwn], zr[kOwn], gr[kOwn];
        auto load_tile = [&](int nt) {
            load4<T, ROWS>(ur, up, offset(a.u), a.u.sl, nt, q);
            load4<T, ROWS>(dr, dp, offset(a.delta), a.delta.sl, nt, q);
            load4<T, ROWS>(gr, gp, offset(ga.dy), ga.dy.sl, nt, q);
            if (gate) load4<T, ROWS>(zr, zp, offset(a.z), a.z.sl, nt, q);
            if (!ENDS) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) hn[nb] = *reinterpret_cast<const float4*>(sv + nb * 16);
            }
            stage_load(nt);
        };
        int nt = end - last;
        load_tile(nt);
        stage_store(lds[0]);
        __syncthreads();
        int buf = 0;
        for (int t0 = last; t0 >= beg; t0 -= kT) {
            float u[kOwn], dt[kOwn], slope[kOwn], dx[kOwn], p[kOwn], zs[kOwn], dyf[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const bool in = step_of<ROWS>(q, i) < nt;
                u[i] = to_f(ur[i]);
                const float v = to_f(dr[i]) + bias;
                slope[i] = 1.0f;
                dt[i] = a.softplus ? softplus_slope_f(v, slope[i]) : v;
                dt[i] = in ? dt[i] : 0.0f;
                dx[i] = dt[i] * u[i];
                dyf[i] = to_f(gr[i]);
                p[i] = dyf[i];
                if (gate) {
                    const float z = to_f(zr[i]), s = sigmoid_f(z);
                    p[i] *= z * s;
                    zs[i] = s * fmaf(z, 1.0f - s, 1.0f);
                }
                p[i] = in && live ? p[i] : 0.0f;  // lanes without a channel add nothing to dB and dC
                if (ENDS) dtsum += dt[i];
            }
            float4 h0v[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) h0v[nb] = hn[nb];
            const int now = nt;
            T *dut = dup, *ddt_to = ddp, *dzt = dzp;
            if (t0 > beg) {
                up -= kT * a.u.sl, dp -= kT * a.delta.sl, zp -= kT * a.z.sl, gp -= kT * ga.dy.sl;
                dup -= kT * ga.du.sl, ddp -= kT * ga.ddelta.sl, dzp -= kT * ga.dz.sl;
                Bp -= kT * a.B.sl, Cp -= kT * a.C.sl, sv -= wstep;
                nt = kT;
                load_tile(nt);
            }
            int bq = buf * kT * kPad + q * 8;  // the lane's B and C in lds
            if constexpr (ENDS) {
#pragma unroll
                for (int t = kT - 1; t >= 0; --t) {
                    const float dtv = quad_bcast(dt[reg<ROWS>(t)], owner<ROWS>(t));
                    const float pv = quad_bcast(p[reg<ROWS>(t)], owner<ROWS>(t));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const float4 c = *reinterpret_cast<const float4*>(&lds[0][0] + bq + t * kPad + nb * 32 + 4);
                        const float cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            carry[nb][j] = fmaf(cv[j], pv, carry[nb][j]) * __builtin_amdgcn_exp2f(dtv * A2[nb][j]);
                    }
                }
            } else {
                float yp[kT], gx[kT], dd[kT];
#pragma unroll
                for (int t = 0; t < kT; ++t) yp[t] = gx[t] = dd[t] = 0.0f;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float dec[kT][4], x[kT + 1][4];
                    x[0][0] = h0v[nb].x, x[0][1] = h0v[nb].y, x[0][2] = h0v[nb].z, x[0][3] = h0v[nb].w;
#pragma unroll
                    for (int t = 0; t < kT; ++t) {
                        const float dtv = quad_bcast(dt[reg<ROWS>(t)], owner<ROWS>(t));
                        const float dxv = quad_bcast(dx[reg<ROWS>(t)], owner<ROWS>(t));
                        const float4 b = *reinterpret_cast<const float4*>(&lds[0][0] + bq + t * kPad + nb * 32);
                        const float4 c = *reinterpret_cast<const float4*>(&lds[0][0] + bq + t * kPad + nb * 32 + 4);
                        const float bv[4] = {b.x, b.y, b.z, b.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            dec[t][j] = __builtin_amdgcn_exp2f(dtv * A2[nb][j]);
                            x[t + 1][j] = fmaf(dec[t][j], x[t][j], dxv * bv[j]);
                            yp[t] = fmaf(cv[j], x[t + 1][j], yp[t]);
                        }
                        asm volatile("" : "+v"(yp[t]));  // the sum is done here, not where it is used
                    }
                    // on the way back B, C and the passed-on values are read anew: kept
                    // from the way forth they would take 10 registers per step
                    asm volatile("" : "+v"(bq));
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) asm volatile("" : "+v"(dt[i]), "+v"(dx[i]));
#pragma unroll
                    for (int t = kT - 1; t >= 0; --t) {
                        const float dtv = quad_bcast(dt[reg<ROWS>(t)], owner<ROWS>(t));
                        const float dxv = quad_bcast(dx[reg<ROWS>(t)], owner<ROWS>(t));
                        const float pv = quad_bcast(p[reg<ROWS>(t)], owner<ROWS>(t));
                        const float4 b = *reinterpret_cast<const float4*>(&lds[0][0] + bq + t * kPad + nb * 32);
                        const float4 c = *reinterpret_cast<const float4*>(&lds[0][0] + bq + t * kPad + nb * 32 + 4);
                        const float bv[4] = {b.x, b.y, b.z, b.w}, cv[4] = {c.x, c.y, c.z, c.w};
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float gt = fmaf(cv[j], pv, carry[nb][j]);
                            v[j] = gt * dxv;
                            v[4 + j] = pv * x[t + 1][j];
                            gx[t] = fmaf(gt, bv[j], gx[t]);
                            carry[nb][j] = gt * dec[t][j];
                            const float back = carry[nb][j] * x[t][j];
                            dd[t] = fmaf(back, A2[nb][j], dd[t]);
                            dA[nb][j] = fmaf(back, dtv, dA[nb][j]);
                        }
                        float s0, s1;
                        channel_sums(v, s0, s1);
                        // [wave][t][nb][B or C][n]: a row of lanes holds two of a kind's four per quad
                        if ((lane & 12) == 0)
                            *reinterpret_cast<float2*>(&red[((wave * kT + t) * NB + nb) * 32 + (lane >> 5) * 16 + q * 4 +
                                                            ((lane >> 4) & 1) * 2]) = make_float2(s0, s1);
                        // these sums are done here too: their operands are a step's registers
                        asm volatile("" : "+v"(gx[t]), "+v"(dd[t]), "+v"(dA[nb][0]), "+v"(dA[nb][1]), "+v"(dA[nb][2]),
                                     "+v"(dA[nb][3]));
                    }
                }
                float ypre[kOwn], gxs[kOwn], dds[kOwn], o[kOwn];
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    constexpr int st = ROWS ? kOwn : 1, mul = ROWS ? 1 : 4;
                    const int t = i * mul;
                    ypre[i] = quad_sums(yp[t], yp[t + st], yp[t + 2 * st], yp[t + 3 * st], odd, high);
                    gxs[i] = quad_sums(gx[t], gx[t + st], gx[t + 2 * st], gx[t + 3 * st], odd, high);
                    dds[i] = quad_sums(dd[t], dd[t + st], dd[t + 2 * st], dd[t + 3 * st], odd, high);
                }
#pragma unroll
                for (int i = 0; i < kOwn; ++i) o[i] = fmaf(Dv, p[i], dt[i] * gxs[i]);
                if (live) store4<T, ROWS>(o, dut, offset(ga.du), ga.du.sl, now, q);
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    o[i] = fmaf(u[i], gxs[i], dds[i] * kLn2) * slope[i];
                    if (step_of<ROWS>(q, i) < now) {
                        dbsum += o[i];
                        dDsum = fmaf(p[i], u[i], dDsum);
                    }
                }
                if (live) store4<T, ROWS>(o, ddt_to, offset(ga.ddelta), ga.ddelta.sl, now, q);
                if (gate) {
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) o[i] = dyf[i] * fmaf(Dv, u[i], ypre[i]) * zs[i];
                    if (live) store4<T, ROWS>(o, dzt, offset(ga.dz), ga.dz.sl, now, q);
                }
                __syncthreads();
                // the workgroup's sums of dB and dC: the four waves' in order
                float* to = sp.part_bc + ((((int64_t)blk * a.Bsz + it.row) * a.q.L + t0) * a.G + g) * (NB * 32);
#pragma unroll
                for (int k = 0; k < NB * 2; ++k) {
                    const int e = tid + 256 * k, t = e / (NB * 32), v = e % (NB * 32);
                    if (t < now) {
                        float s = red[e];
#pragma unroll
                        for (int w = 1; w < 4; ++w) s += red[w * kT * NB * 32 + e];
                        to[(int64_t)t * a.G * (NB * 32) + v] = s;
                    }
                }
            }
            if (t0 > beg) {
                buf ^= 1;
                stage_store(lds[buf]);
                __syncthreads();
            }
        }
    }

    if (ENDS) {
        dtsum += dpp<0xB1>(dtsum);
        dtsum += dpp<0x4E>(dtsum);
        if (live) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                *reinterpret_cast<float4*>(sp.ends + item * wstep + wrow + nb * 16) =
                    make_float4(carry[nb][0], carry[nb][1], carry[nb][2], carry[nb][3]);
            if (q == 0) sp.sums[item * a.H + h0] = dtsum;
        }
        return;
    }
    dDsum += dpp<0xB1>(dDsum);
    dDsum += dpp<0x4E>(dDsum);
    dbsum += dpp<0xB1>(dbsum);
    dbsum += dpp<0x4E>(dbsum);
    if (!live) return;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
        *reinterpret_cast<float4*>(sp.part_a + item * wstep + wrow + nb * 16) =
            make_float4(dA[nb][0], dA[nb][1], dA[nb][2], dA[nb][3]);
    if (q == 0) {
        sp.part_d[(item * 2) * a.H + h0] = dDsum;
        sp.part_d[(item * 2 + 1) * a.H + h0] = dbsum;
    }
    if (work && it.c == 0 && ga.dx_in) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = nb * 16 + q * 4 + j;
                if (n < N) ga.dx_in[((int64_t)it.s * a.H + h0) * N + n] = carry[nb][j];
            }
    }
}

// dB and dC from the workgroups' sums; steps outside every sequence stay as they were
template <class T>
__global__ __launch_bounds__(256) void grad_bc_kernel(ScanGradArgs ga, const float* part, int per_group, int NB) {
    const ScanArgs& a = ga.f;
    const int64_t row = (int64_t)NB * 32, total = a.Bsz * a.q.L * a.G * row;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int v = (int)(i % row);
    const int g = (int)(i / row % a.G);
    const int64_t bl = i / (row * a.G);
    const int64_t b = bl / a.q.L;
    const int t = (int)(bl % a.q.L), n = (v >> 5) * 16 + (v & 15);
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
        if (Q < 4 * kT) Q = 4 * kT;
    }
    Q = (Q + kT - 1) / kT * kT;
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

template <class T, int NB, bool ROWS>
hipError_t launch_as(const ScanGradArgs& g, const Plan& p, hipStream_t s) {
    const ScanArgs& a = g.f;
    const int64_t wgs = p.items * p.sp.blocks;
    const int64_t bc = (a.Bsz * a.q.L * a.G * NB * 32 + 255) / 256;
    if (wgs >= ((int64_t)1 << 31) || bc >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), wg(256);
    if (p.split) grad_kernel<T, NB, ROWS, true><<<grid, wg, 0, s>>>(g, p.sp);
    grad_kernel<T, NB, ROWS, false><<<grid, wg, 0, s>>>(g, p.sp);
    grad_bc_kernel<T><<<dim3((unsigned)bc), wg, 0, s>>>(g, p.sp.part_bc, p.sp.per_group, NB);
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
    if (N <= 16) return rows ? launch_as<T, 1, true>(g, p, s) : launch_as<T, 1, false>(g, p, s);
    if (N <= 32) return rows ? launch_as<T, 2, true>(g, p, s) : launch_as<T, 2, false>(g, p, s);
    return rows ? launch_as<T, 4, true>(g, p, s) : launch_as<T, 4, false>(g, p, s);
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

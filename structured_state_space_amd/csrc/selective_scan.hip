// Selective state-space scan, forward:
//   dt = softplus(delta + delta_bias)
//   x_t[n] = exp(dt_t A[n]) x_{t-1}[n] + dt_t u_t B_t[n]
//   y_t = (sum_n C_t[n] x_t[n] + D u_t) silu(z_t)
// per (sequence, channel), B and C shared by the channels of a group.
//
// Work split.  A quad of lanes holds one channel's states (lane q the states
// 16 nb + 4 q + j), a wave 16 channels, a workgroup 64 channels of one group.
// The steps run in order, 32 to a tile: lane q loads and prepares (softplus,
// gate) 8 of the tile's steps and the quad passes dt and dt u around with
// quad_perm; B and C of a tile go through LDS in float32, double-buffered, the
// next tile's loads in flight while this one is computed.
//
// Where channels and sequences alone leave the GPU idle, the steps are split
// into chunks of Q as well: a first launch computes every chunk's state from a
// zero start (without C and y) and the sum of its dt, whose exp(A sum dt) is
// the chunk's whole decay; in the second each chunk folds its predecessors'
// ends into its start state and runs the full recurrence.
#include "selective.hpp"

namespace ssm {

namespace {

constexpr int kTile = 32;
constexpr int kChannels = 64;  // per workgroup

// step t of a tile is owned by quad lane owner(t), in its register reg(t)
template <bool ROWS>
constexpr int owner(int t) { return ROWS ? t >> 3 : t & 3; }
template <bool ROWS>
constexpr int reg(int t) { return ROWS ? t & 7 : t >> 2; }
template <bool ROWS>
__device__ __forceinline__ int step_of(int q, int r) { return ROWS ? q * 8 + r : r * 4 + q; }

// the 8 steps of a tile that lane q owns; `base` is the same in the whole wave
// (the tile's first step, the wave's first channel), `off` is the lane's
// offset from it: its channel and its first step
template <class T, bool ROWS>
__device__ __forceinline__ void load8(T (&r)[8], const T* base, uint32_t off, int64_t sl, int nt, int q) {
    if (nt == kTile) {
        if constexpr (ROWS) {
            const Vec8<T> v = *reinterpret_cast<const Vec8<T>*>(base + off);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = v.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i, base += 4 * sl) r[i] = base[off];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i, base += ROWS ? 1 : 4 * sl)
            r[i] = step_of<ROWS>(q, i) < nt ? base[off] : from_f<T>(0.0f);
    }
}

template <class T, bool ROWS>
__device__ __forceinline__ void store8(const float (&v)[8], T* base, uint32_t off, int64_t sl, int nt, int q) {
    if (nt == kTile) {
        if constexpr (ROWS) {
            Vec8<T> w;
#pragma unroll
            for (int i = 0; i < 8; ++i) w.v[i] = from_f<T>(v[i]);
            *reinterpret_cast<Vec8<T>*>(base + off) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i, base += 4 * sl) base[off] = from_f<T>(v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i, base += ROWS ? 1 : 4 * sl)
            if (step_of<ROWS>(q, i) < nt) base[off] = from_f<T>(v[i]);
    }
}

// what a launch of scan_kernel is for
enum Mode {
    kEnds,    // every chunk's end state from a zero start, and its sum of dt
    kFull,    // y, and the final and saved states where asked for
    kStates,  // the saved states alone
};

// one tile's recurrence; GUARD: only the first nt steps exist (a branch per step)
template <int NB, bool ROWS, Mode MODE, bool GUARD>
__device__ __forceinline__ void run_tile(float (&h)[NB][4], const float (&A2)[NB][4], const float (&dt)[8],
                                         const float (&dx)[8], const float* lds, int pad, int q, int nt,
                                         float (&p)[kTile], float* saved, int64_t saved_step) {
#pragma unroll
    for (int t = 0; t < kTile; ++t) {
        if (GUARD && t >= nt) continue;
        if (MODE != kEnds && t % kSaveSteps == 0 && saved) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                *reinterpret_cast<float4*>(saved + (t / kSaveSteps) * saved_step + nb * 16) =
                    make_float4(h[nb][0], h[nb][1], h[nb][2], h[nb][3]);
        }
        const float dtv = quad_bcast(dt[reg<ROWS>(t)], owner<ROWS>(t));
        const float dxv = quad_bcast(dx[reg<ROWS>(t)], owner<ROWS>(t));
        float acc = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const float4 b = *reinterpret_cast<const float4*>(lds + t * pad + (nb * 4 + q) * 8);
            const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[nb][j] = fmaf(__builtin_amdgcn_exp2f(dtv * A2[nb][j]), h[nb][j], dxv * bv[j]);
            if (MODE == kFull) {
                const float4 c = *reinterpret_cast<const float4*>(lds + t * pad + (nb * 4 + q) * 8 + 4);
                const float cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = fmaf(cv[j], h[nb][j], acc);
            }
        }
        // the sum is done here: left alone, the compiler moves the sums of the two
        // forms of this loop behind both of them and holds every step's states
        // (hundreds of registers)
        if (MODE == kFull) asm volatile("" : "+v"(acc));
        p[t] = acc;
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

template <class T, int NB, bool ROWS, Mode MODE>
__global__ __launch_bounds__(256, NB == 1 ? 3 : 2) void scan_kernel(ScanArgs a, Split sp) {
    constexpr bool ENDS = MODE == kEnds, FULL = MODE == kFull;
    constexpr int kPad = NB * 32 + 4;
    constexpr int kStage = NB * 2;  // elements of B (and of C) that a thread stages per tile
    __shared__ __attribute__((aligned(16))) float lds[2][kTile * kPad];

    const int cb = blockIdx.x % sp.blocks;
    const int64_t item = blockIdx.x / sp.blocks;
    Item it;
    if (!find_item(a.q, item, sp.Q, it) || it.state < 0) return;
    const int beg = it.beg + it.c * sp.Q;
    const int end = min((int64_t)it.end, (int64_t)beg + sp.Q);
    const int chunks = chunks_of(it.end - it.beg, sp.Q);
    if (it.c >= chunks || (ENDS && it.c + 1 == chunks)) return;

    const int tid = threadIdx.x, lane = tid & 63, q = lane & 3;
    const bool odd = q & 1, high = q & 2;
    const int Hg = (int)(a.H / a.G), N = (int)a.N, Np = NB * 16;
    const int g = cb / sp.per_group;
    const int c0 = (cb % sp.per_group) * kChannels + __builtin_amdgcn_readfirstlane(tid >> 6) * 16;  // wave's first channel in the group
    const int lc = lane >> 2;
    const bool live = c0 + lc < Hg;
    const int w0 = g * Hg + min(c0, Hg - 1);             // wave's first channel, clamped
    const int h0 = g * Hg + min(c0 + lc, Hg - 1);        // the lane's
    const uint32_t dh = (uint32_t)(h0 - w0);

    float A2[NB][4], h[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = nb * 16 + q * 4 + j;
            A2[nb][j] = n < N ? a.A[(int64_t)h0 * N + n] * kLog2e : 0.0f;
            h[nb][j] = 0.0f;
        }
    const float bias = a.delta_bias ? a.delta_bias[h0] : 0.0f;
    const float Dv = a.D ? a.D[h0] : 0.0f;
    const int64_t wrow = ((int64_t)h0) * Np + q * 4;      // in a workspace row [H, Np]
    const int64_t wstep = a.H * Np;

    // start state
    if (it.c == 0) {
        if (!ENDS && sp.starts) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float4 v = *reinterpret_cast<const float4*>(sp.starts + it.s * wstep + wrow + nb * 16);
                h[nb][0] = v.x, h[nb][1] = v.y, h[nb][2] = v.z, h[nb][3] = v.w;
            }
        }
        if (ENDS || !sp.starts || chunks == 1) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = nb * 16 + q * 4 + j;
                    h[nb][j] = a.x_in && n < N ? a.x_in[(it.state * a.H + h0) * N + n] : 0.0f;
                }
        }
        if (ENDS && live) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                *reinterpret_cast<float4*>(sp.starts + it.s * wstep + wrow + nb * 16) =
                    make_float4(h[nb][0], h[nb][1], h[nb][2], h[nb][3]);
        }
    } else if (!ENDS) {
        const int64_t first = item - it.c;
        for (int64_t i = first; i < item; ++i) {
            const float s = i == first ? 0.0f : sp.sums[i * a.H + h0];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float4 v = *reinterpret_cast<const float4*>(sp.ends + i * wstep + wrow + nb * 16);
                const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[nb][j] = i == first ? e[j] : fmaf(__builtin_amdgcn_exp2f(s * A2[nb][j]), h[nb][j], e[j]);
            }
        }
    }

    // wave-uniform bases at the tile's first step; lane offsets
    const T* up = (const T*)a.u.data + it.row * a.u.sb + w0 * a.u.sh + beg * a.u.sl;
    const T* dp = (const T*)a.delta.data + it.row * a.delta.sb + w0 * a.delta.sh + beg * a.delta.sl;
    const T* zp = (const T*)a.z.data + it.row * a.z.sb + w0 * a.z.sh + beg * a.z.sl;
    T* yp = (T*)a.y.data + it.row * a.y.sb + w0 * a.y.sh + beg * a.y.sl;
    const uint32_t q0 = ROWS ? q * 8 : q;  // the lane's first step
    const uint32_t uo = dh * (uint32_t)a.u.sh + q0 * (uint32_t)a.u.sl;
    const uint32_t dof = dh * (uint32_t)a.delta.sh + q0 * (uint32_t)a.delta.sl;
    const uint32_t zo = dh * (uint32_t)a.z.sh + q0 * (uint32_t)a.z.sl;
    const uint32_t yo = dh * (uint32_t)a.y.sh + q0 * (uint32_t)a.y.sl;
    const bool gate = FULL && a.z.data;

    const T* Bp = (const T*)a.B.data + it.row * a.B.sb + g * a.B.sg + beg * a.B.sl;
    const T* Cp = (const T*)a.C.data + it.row * a.C.sb + g * a.C.sg + beg * a.C.sl;
    const bool by_time = a.B.sl == 1;  // staging order: consecutive threads along B's contiguous axis
    T sb[kStage], sc[kStage];
    auto stage_pos = [&](int k, int& t, int& n) {
        const int e = tid + 256 * k;
        t = by_time ? e % kTile : e / (NB * 16);
        n = by_time ? e / kTile : e % (NB * 16);
    };
    auto stage_load = [&](int nt) {
#pragma unroll
        for (int k = 0; k < kStage; ++k) {
            int t, n;
            stage_pos(k, t, n);
            const bool in = t < nt && n < N;
            sb[k] = in ? Bp[(uint32_t)n * (uint32_t)a.B.sn + (uint32_t)t * (uint32_t)a.B.sl] : from_f<T>(0.0f);
            if (FULL)
                sc[k] = in ? Cp[(uint32_t)n * (uint32_t)a.C.sn + (uint32_t)t * (uint32_t)a.C.sl] : from_f<T>(0.0f);
        }
    };
    auto stage_store = [&](float* to) {
#pragma unroll
        for (int k = 0; k < kStage; ++k) {
            int t, n;
            stage_pos(k, t, n);
            float* at = to + t * kPad + (n >> 2) * 8 + (n & 3);
            at[0] = to_f(sb[k]);
            if (FULL) at[4] = to_f(sc[k]);
        }
    };

    T ur[8], dr[8], zr[8];
    int nt = min(kTile, end - beg);
    if (nt > 0) {
        load8<T, ROWS>(ur, up, uo, a.u.sl, nt, q);
        load8<T, ROWS>(dr, dp, dof, a.delta.sl, nt, q);
        if (gate) load8<T, ROWS>(zr, zp, zo, a.z.sl, nt, q);
        stage_load(nt);
        stage_store(lds[0]);
        __syncthreads();
    }
    float sum = 0.0f;
    float* saved = !ENDS && a.saved && live
                       ? a.saved + (saved_row(a.q, it) + (beg - it.beg) / kSaveSteps) * wstep + wrow
                       : nullptr;
    const bool saving = !ENDS && a.saved;
    int buf = 0;
    for (int t0 = beg; t0 < end; t0 += kTile) {
        float dt[8], dx[8], uf[8], zf[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uf[i] = to_f(ur[i]);
            if (gate) zf[i] = to_f(zr[i]);
            const float v = to_f(dr[i]) + bias;
            dt[i] = a.softplus ? softplus_f(v) : v;
            dx[i] = dt[i] * uf[i];
            if (ENDS) sum += step_of<ROWS>(q, i) < nt ? dt[i] : 0.0f;
        }
        const int now = nt, next = min(kTile, end - t0 - kTile);
        T* yt = yp;
        if (next > 0) {
            up += kTile * a.u.sl, dp += kTile * a.delta.sl, zp += kTile * a.z.sl, yp += kTile * a.y.sl;
            Bp += kTile * a.B.sl, Cp += kTile * a.C.sl;
            load8<T, ROWS>(ur, up, uo, a.u.sl, next, q);
            load8<T, ROWS>(dr, dp, dof, a.delta.sl, next, q);
            if (gate) load8<T, ROWS>(zr, zp, zo, a.z.sl, next, q);
            stage_load(next);
        }
        float p[kTile];
        if (now == kTile) {
            run_tile<NB, ROWS, MODE, false>(h, A2, dt, dx, lds[buf], kPad, q, now, p, saved, wstep);
        } else {
#pragma unroll
            for (int t = 0; t < kTile; ++t) p[t] = 0.0f;
            run_tile<NB, ROWS, MODE, true>(h, A2, dt, dx, lds[buf], kPad, q, now, p, saved, wstep);
        }
        if (saving && live) saved += (kTile / kSaveSteps) * wstep;
        if (FULL) {
            float yv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = ROWS ? quad_sums(p[i], p[8 + i], p[16 + i], p[24 + i], odd, high)
                                     : quad_sums(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3], odd, high);
                yv[i] = fmaf(Dv, uf[i], s);
                if (gate) yv[i] *= silu_f(zf[i]);
            }
            if (live) store8<T, ROWS>(yv, yt, yo, a.y.sl, now, q);
        }
        if (next > 0) {
            buf ^= 1;
            stage_store(lds[buf]);
            __syncthreads();
            nt = next;
        }
    }

    if (ENDS) {
        sum += dpp<0xB1>(sum);
        sum += dpp<0x4E>(sum);
        if (live) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                *reinterpret_cast<float4*>(sp.ends + item * wstep + wrow + nb * 16) =
                    make_float4(h[nb][0], h[nb][1], h[nb][2], h[nb][3]);
            if (q == 0) sp.sums[item * a.H + h0] = sum;
        }
    } else if (live && a.x_out && it.c + 1 == chunks) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = nb * 16 + q * 4 + j;
                if (n < N) a.x_out[(it.state * a.H + h0) * N + n] = h[nb][j];
            }
    }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
    Split sp;
    int64_t items;
    bool split;
    size_t ends_bytes, sums_bytes, starts_bytes;
};

// Chunks are made where channels and sequences give fewer than kFew
// workgroups (a packed batch: always, its sequences may be one long one), and
// then so that about kMany workgroups share the steps.
Plan plan(const Seqs& q, int64_t H, int64_t N, int64_t G) {
    constexpr int64_t kFew = 192, kMany = 512;
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
    p.items = item_count(q, Q);
    const size_t Np = (size_t)padded_states(N);
    p.ends_bytes = p.split ? up256((size_t)p.items * H * Np * 4) : 0;
    p.sums_bytes = p.split ? up256((size_t)p.items * H * 4) : 0;
    p.starts_bytes = p.split ? up256((size_t)q.S * H * Np * 4) : 0;
    return p;
}

template <class T, int NB, bool ROWS>
hipError_t launch_as(const ScanArgs& a, const Plan& p, hipStream_t s) {
    const int64_t wgs = p.items * p.sp.blocks;
    if (wgs >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    if (p.split) scan_kernel<T, NB, ROWS, kEnds><<<dim3((unsigned)wgs), dim3(256), 0, s>>>(a, p.sp);
    if (a.y.data)
        scan_kernel<T, NB, ROWS, kFull><<<dim3((unsigned)wgs), dim3(256), 0, s>>>(a, p.sp);
    else
        scan_kernel<T, NB, ROWS, kStates><<<dim3((unsigned)wgs), dim3(256), 0, s>>>(a, p.sp);
    return hipGetLastError();
}

template <class T>
hipError_t launch_of(const ScanArgs& a, const Plan& p, bool rows, hipStream_t s) {
    if (a.N <= 16) return rows ? launch_as<T, 1, true>(a, p, s) : launch_as<T, 1, false>(a, p, s);
    if (a.N <= 32) return rows ? launch_as<T, 2, true>(a, p, s) : launch_as<T, 2, false>(a, p, s);
    return rows ? launch_as<T, 4, true>(a, p, s) : launch_as<T, 4, false>(a, p, s);
}

}  // namespace

size_t scan_workspace_bytes(const Seqs& q, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, H, N, G);
    return p.ends_bytes + p.sums_bytes + p.starts_bytes;
}

bool scan_fits(const Seqs& q, int64_t H, int64_t N, int64_t G) {
    const Plan p = plan(q, H, N, G);
    return p.items * p.sp.blocks < ((int64_t)1 << 31);
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
    // steps contiguous in every tensor: the vector loads and stores of "rows"
    const bool rows = a.u.sl == 1 && a.delta.sl == 1 && (!a.z.data || a.z.sl == 1) && (!a.y.data || a.y.sl == 1);
    if (dtype == SSM_F32) return launch_of<float>(a, p, rows, s);
    if (dtype == SSM_BF16) return launch_of<bf16>(a, p, rows, s);
    return launch_of<f16>(a, p, rows, s);
}

}  // namespace ssm

// Selective state-space scan, forward:
//   dt = softplus(delta + delta_bias)
//   x_t[n] = exp(dt_t A[n]) x_{t-1}[n] + dt_t u_t B_t[n]
//   y_t = (sum_n C_t[n] x_t[n] + D u_t) silu(z_t)
// per (sequence, channel), B and C shared by the channels of a group.
//
// Work split.  Eight lanes share a channel, a wave has 8 channels, a workgroup 64
// of one group.  The steps run in order, 32 to a tile: each lane loads and
// prepares (softplus, gate) four of a tile's steps, and the channel's lanes pass
// dt and dt u around by DPP; B and C of a tile go through LDS in float32,
// double-buffered, the next tile's loads in flight while this one is computed.
//
// Where channels and sequences alone leave the GPU idle, the steps are split
// into chunks of Q as well: a first launch computes every chunk's state from a
// zero start (without C and y) and the sum of its dt, whose exp(A sum dt) is
// the chunk's whole decay; in the second each chunk folds its predecessors'
// ends into its start state and runs the full recurrence.
#include "selective.hpp"

namespace ssm {

namespace {

// what a launch of scan_kernel is for
enum Mode {
    kEnds,    // every chunk's end state from a zero start, and its sum of dt
    kFull,    // y, and the final and saved states where asked for
    kStates,  // the saved states alone
};

// one tile's recurrence; GUARD: only the first nt steps exist (a branch per step).
// B and C come from LDS a pair of steps ahead of their use.
template <int S, bool ROWS, Mode MODE, bool GUARD>
__device__ __forceinline__ void run_tile(float (&h)[S], const float (&A2)[S], const float (&dt)[2][kOwn],
                                         const float (&dx)[2][kOwn], const float* lds, int nt, bool odd, bool high,
                                         float (&sums)[2][kOwn]) {
    constexpr int kRow = Stage<float, S>::kRow, kGroup = S == 2 ? 4 : S == 4 ? 2 : 1;
    float4 bc[2][kGroup][S / 2];
    float p[ROWS ? 16 : 4];  // the lanes' shares of y, until a quad's four owners have one each
    auto fetch = [&](int g) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
            for (int k = 0; k < S / 2; ++k)
                bc[g & 1][i][k] = *reinterpret_cast<const float4*>(lds + (g * kGroup + i) * kRow + k * 32);
    };
    auto collect = [&](int t) {  // after step t
        if (MODE != kFull) return;
        if (!ROWS && (t & 3) == 3) sums[t >> 4][(t >> 2) & 3] = quad_sums(p[0], p[1], p[2], p[3], odd, high);
        if (ROWS && (t & 15) == 15) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                sums[t >> 4][i] = quad_sums(p[i], p[(4 + i) & 15], p[(8 + i) & 15], p[(12 + i) & 15], odd, high);
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
            float& share = p[ROWS ? t & 15 : t & 3];
            if (GUARD && t >= nt) {
                share = 0.0f;
                collect(t);
                continue;
            }
            const float dtv = quad_bcast(dt[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
            const float dxv = quad_bcast(dx[t >> 4][reg<ROWS>(t)], pos<ROWS>(t));
            float acc = 0.0f;
#pragma unroll
            for (int k = 0; k < S / 2; ++k) {
                const float4 v = bc[g & 1][i][k];
                h[2 * k] = fmaf(__builtin_amdgcn_exp2f(dtv * A2[2 * k]), h[2 * k], dxv * v.x);
                h[2 * k + 1] = fmaf(__builtin_amdgcn_exp2f(dtv * A2[2 * k + 1]), h[2 * k + 1], dxv * v.y);
                if (MODE == kFull) acc = fmaf(v.w, h[2 * k + 1], fmaf(v.z, h[2 * k], acc));
            }
            // the sum is done here: left alone, the compiler moves the sums of the two
            // forms of this loop behind both of them and holds every step's states
            // (hundreds of registers)
            if (MODE == kFull) asm volatile("" : "+v"(acc));
            share = acc;
            collect(t);
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

template <class T, int S, bool ROWS, Mode MODE>
__global__ __launch_bounds__(kScanThreads, S <= 4 ? 4 : 2) void scan_kernel(ScanArgs a, Split sp) {
    constexpr bool ENDS = MODE == kEnds, FULL = MODE == kFull;
    using St = Stage<T, S>;
    __shared__ __attribute__((aligned(16))) float lds[2][kTile * St::kRow];

    const int cb = blockIdx.x % sp.blocks;
    const int64_t item = blockIdx.x / sp.blocks;
    Item it;
    if (!find_item(a.q, item, sp.Q, it) || it.state < 0) return;
    const int beg = it.beg + it.c * sp.Q;
    const int end = min((int64_t)it.end, (int64_t)beg + sp.Q);
    const int chunks = chunks_of(it.end - it.beg, sp.Q);
    if (it.c >= chunks || (ENDS && it.c + 1 == chunks)) return;

    const Place l = place_of(cb, sp.per_group, a.H, a.G);
    const int p = l.p, N = (int)a.N;
    const bool odd = p & 1, high = p & 2, upper = p & 4;
    float A2[S], h[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        A2[j] = p * S + j < N ? a.A[(int64_t)l.h * N + p * S + j] * kLog2e : 0.0f;
        h[j] = 0.0f;
    }
    const float bias = a.delta_bias ? a.delta_bias[l.h] : 0.0f;
    const float Dv = a.D ? a.D[l.h] : 0.0f;
    const int64_t wrow = (int64_t)l.h * (8 * S) + p * S;  // in a workspace row [H, Np]
    const int64_t wstep = a.H * (8 * S);

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
#pragma unroll
            for (int j = 0; j < S; ++j) h[j] = fmaf(__builtin_amdgcn_exp2f(s * A2[j]), h[j], e[j]);
        }
    }

    // bases at the tile's first step, the same in the whole wave, and the lanes'
    // distances from them in bytes (the strides' limits keep these below 2^32)
    constexpr uint32_t kE = sizeof(T);
    const uint32_t q0 = step_of<ROWS>(p, 0);
    auto base = [&](const View3& v) {
        return (char*)v.data + (it.row * v.sb + l.w0 * v.sh + beg * v.sl) * (int64_t)kE;
    };
    auto offset = [&](const View3& v) { return (l.dh * (uint32_t)v.sh + q0 * (uint32_t)v.sl) * kE; };
    const bool gate = FULL && a.z.data;
    const View3& gv = gate ? a.z : a.u;  // without a gate u once more, unused: the loads need no branch
    const char *up = base(a.u), *dp = base(a.delta), *zp = base(gv);
    char* yp = base(a.y);
    const uint32_t uo = offset(a.u), dof = offset(a.delta), zo = offset(gv), yo = offset(a.y);
    const uint32_t us = (uint32_t)a.u.sl * 4 * kE, ds = (uint32_t)a.delta.sl * 4 * kE,
                   zs = (uint32_t)gv.sl * 4 * kE, ys = (uint32_t)a.y.sl * 4 * kE;
    const char* Bp = (const char*)a.B.data + (it.row * a.B.sb + l.g * a.B.sg + beg * a.B.sl) * (int64_t)kE;
    const char* Cp = (const char*)a.C.data + (it.row * a.C.sb + l.g * a.C.sg + beg * a.C.sl) * (int64_t)kE;
    const uint32_t bs = (uint32_t)a.B.sl * 4 * kE, cs = (uint32_t)a.C.sl * 4 * kE;
    St stage;
    stage.init(a.B, a.C, N, l.tid);

    T ur[kOwn], dr[kOwn], zr[kOwn];
    auto load_tile = [&]() {
        load_own<T, ROWS>(ur, up, uo, us);
        load_own<T, ROWS>(dr, dp, dof, ds);
        if (FULL) load_own<T, ROWS>(zr, zp, zo, zs);
        stage.template load<true, FULL>(Bp, Cp);
    };
    auto advance = [&](uint32_t go) {  // by 4 go steps
        up += (uint64_t)us * go, dp += (uint64_t)ds * go, zp += (uint64_t)zs * go;
        Bp += (uint64_t)bs * go, Cp += (uint64_t)cs * go;
    };
    float dt[2][kOwn], dx[2][kOwn], uf[kOwn], zf[kOwn], sum = 0.0f;
    auto prepare = [&](int nt) {  // the lane's own steps, then all of the channel's
        float d[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            uf[i] = to_f(ur[i]);
            if (FULL) zf[i] = to_f(zr[i]);
            d[i] = to_f(dr[i]) + bias;
        }
        if (a.softplus) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) d[i] = softplus_f<kFine<T>>(d[i]);
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (ENDS) sum += step_of<ROWS>(p, i) < nt ? d[i] : 0.0f;
            both_halves(d[i], dt[0][i], dt[1][i]);
            both_halves(d[i] * uf[i], dx[0][i], dx[1][i]);
        }
    };
    auto finish = [&](const float (&s)[2][kOwn], int nt) {  // y of the lane's own steps
        float yv[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) yv[i] = fmaf(Dv, uf[i], half_sums(s[0][i], s[1][i], upper));
        if (gate) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) yv[i] *= silu_f<kFine<T>>(zf[i]);
        }
        if (l.live) store_own<T, ROWS>(yv, yp, yo, ys, nt, p);
    };

    float* saved = !ENDS && a.saved && l.live
                       ? a.saved + (saved_row(a.q, it) + (beg - it.beg) / kTile) * wstep + wrow
                       : nullptr;
    const int whole = max(0, end - beg) / kTile, rest = max(0, end - beg) % kTile;
    int buf = 0;
    if (whole > 0) {
        load_tile();
        stage.template store<true, FULL>(lds[0]);
        __syncthreads();
    }
    for (int k = 0; k < whole; ++k) {
        prepare(kTile);
        // the next whole tile's loads fly while this one is computed (the last one
        // loads itself again: a branch here would make them wait)
        advance(k + 1 < whole ? kTile / 4 : 0);
        load_tile();
        __builtin_amdgcn_sched_barrier(0);  // left alone, the compiler moves the loads behind the tile
        if (saved) {
            store_states<S>(h, saved);
            saved += wstep;
        }
        float s[2][kOwn];
        run_tile<S, ROWS, MODE, false>(h, A2, dt, dx, lds[buf] + p * 4, kTile, odd, high, s);
        if (FULL) finish(s, kTile);
        yp += (uint64_t)ys * (kTile / 4);
        buf ^= 1;
        stage.template store<true, FULL>(lds[buf]);
        __syncthreads();
    }
    if (rest > 0) {
        if (whole > 0) advance(kTile / 4);
        load_part<T, ROWS>(ur, up, uo, us, rest, p);
        load_part<T, ROWS>(dr, dp, dof, ds, rest, p);
        if (FULL) load_part<T, ROWS>(zr, zp, zo, zs, rest, p);
        stage.template load_part<true, FULL>(Bp, Cp, rest);
        buf ^= 1;
        stage.template store<true, FULL>(lds[buf]);
        __syncthreads();
        prepare(rest);
        if (saved) store_states<S>(h, saved);
        float s[2][kOwn];
        run_tile<S, ROWS, MODE, true>(h, A2, dt, dx, lds[buf] + p * 4, rest, odd, high, s);
        if (FULL) finish(s, rest);
    }

    if (ENDS) {
        sum = lane_sum(sum);
        if (l.live) {
            store_states<S>(h, sp.ends + item * wstep + wrow);
            if (p == 0) sp.sums[item * a.H + l.h] = sum;
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

template <class T, int S, bool ROWS>
hipError_t launch_as(const ScanArgs& a, const Plan& p, hipStream_t s) {
    const int64_t wgs = p.items * p.sp.blocks;
    if (wgs >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    if (p.split) scan_kernel<T, S, ROWS, kEnds><<<dim3((unsigned)wgs), dim3(kScanThreads), 0, s>>>(a, p.sp);
    if (a.y.data)
        scan_kernel<T, S, ROWS, kFull><<<dim3((unsigned)wgs), dim3(kScanThreads), 0, s>>>(a, p.sp);
    else
        scan_kernel<T, S, ROWS, kStates><<<dim3((unsigned)wgs), dim3(kScanThreads), 0, s>>>(a, p.sp);
    return hipGetLastError();
}

template <class T>
hipError_t launch_of(const ScanArgs& a, const Plan& p, bool rows, hipStream_t s) {
    if (a.N <= 16) return rows ? launch_as<T, 2, true>(a, p, s) : launch_as<T, 2, false>(a, p, s);
    if (a.N <= 32) return rows ? launch_as<T, 4, true>(a, p, s) : launch_as<T, 4, false>(a, p, s);
    return rows ? launch_as<T, 8, true>(a, p, s) : launch_as<T, 8, false>(a, p, s);
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

// C ABI entry points of the selective operators: argument checks and launches.
#include <string.h>

#include "selective.hpp"

namespace ssm {
size_t scan_workspace_bytes(const Seqs& q, int64_t H, int64_t N, int64_t G);
bool scan_fits(const Seqs& q, int64_t H, int64_t N, int64_t G);
hipError_t launch_scan(int dtype, const ScanArgs& a, void* ws, hipStream_t s);
size_t scan_grad_workspace_bytes(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G);
bool scan_grad_fits(const Seqs& q, int64_t Bsz, int64_t H, int64_t N, int64_t G);
hipError_t launch_scan_backward(int dtype, const ScanGradArgs& g, void* ws, hipStream_t s);
size_t conv_grad_workspace_bytes(const Seqs& q, int64_t H, int width);
bool conv_fits(const Seqs& q, int64_t H);
hipError_t launch_causal_conv(int dtype, const ConvArgs& a, hipStream_t s);
hipError_t launch_causal_conv_backward(int dtype, const ConvGradArgs& g, void* ws, hipStream_t s);
hipError_t launch_selective_step(int dtype, const StepArgs& a, hipStream_t s);
hipError_t launch_causal_conv_step(int dtype, const ConvStepArgs& a, hipStream_t s);
}  // namespace ssm

using namespace ssm;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxStates = 64;
constexpr int64_t kMaxWidth = 4;
// a thread's distance from its workgroup's first channel (or state) and step is
// 32 bits wide in bytes: up to 67 channels or 64 states, and 32 steps, of 4 bytes
constexpr int64_t kMaxStride = (int64_t)1 << 23;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool type_known(int dtype) { return dtype == SSM_F32 || dtype == SSM_BF16 || dtype == SSM_F16; }
size_t type_bytes(int dtype) { return dtype == SSM_F32 ? 4 : 2; }
int device_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_DEVICE; }

// sizes of a call on whole sequences
int check_sizes(int64_t Bsz, int64_t H, int64_t L, int64_t S, bool packed) {
    if (Bsz < 1 || H < 1 || L < 1 || S < 1 || (packed ? Bsz != 1 : S != Bsz)) return SSM_ERR_INVALID_ARGUMENT;
    if (Bsz >= kMaxDim || H >= kMaxDim || L >= kMaxDim - 64 || S >= kMaxDim - 64 || Bsz * H >= kMaxDim ||
        S * H >= kMaxDim || Bsz * H > ((int64_t)1 << 40) / L)
        return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int check_scan_sizes(int64_t H, int64_t N, int64_t G) {
    if (N < 1 || G < 1 || H % G != 0) return SSM_ERR_INVALID_ARGUMENT;
    return N > kMaxStates ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

int check_sequences(const ssm_sequences* q, int64_t H, bool slots_allowed, Seqs* out) {
    if (!q) return SSM_ERR_INVALID_ARGUMENT;
    const int rc = check_sizes(q->Bsz, H, q->L, q->S, q->offsets != nullptr);
    if (rc != SSM_OK) return rc;
    if (q->offsets && q->lengths) return SSM_ERR_INVALID_ARGUMENT;
    if (q->slots && (!slots_allowed || q->n_slots < 1)) return SSM_ERR_INVALID_ARGUMENT;
    if (!aligned(q->offsets, 4) || !aligned(q->lengths, 4) || !aligned(q->slots, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (q->slots && q->n_slots > ((int64_t)1 << 40) / H) return SSM_ERR_UNSUPPORTED;
    out->S = q->S;
    out->L = q->L;
    out->offsets = q->offsets;
    out->lengths = q->lengths;
    out->slots = q->slots;
    out->n_slots = q->n_slots;
    return SSM_OK;
}

Seqs sequences_of(int64_t L, int64_t S, bool packed) {
    Seqs q;
    q.S = S;
    q.L = L;
    q.offsets = packed ? reinterpret_cast<const int32_t*>(16) : nullptr;  // only tested for null by the size rules
    return q;
}

// an output's dimensions of more than one element must not be broadcast
bool strides_fit(int64_t sb, int64_t sh, int64_t sl) {
    return sb < ((int64_t)1 << 40) && sh < kMaxStride && sl < kMaxStride;
}

int check_view(const ssm_view* v, int dtype, bool required, bool output, const ssm_sequences* q, int64_t H) {
    if (!v || !v->data) return required ? SSM_ERR_INVALID_ARGUMENT : SSM_OK;
    if (!aligned(v->data, type_bytes(dtype)) || v->sb < 0 || v->sh < 0 || v->sl < 0) return SSM_ERR_INVALID_ARGUMENT;
    if (output && ((v->sb == 0 && q->Bsz > 1) || (v->sh == 0 && H > 1) || (v->sl == 0 && q->L > 1)))
        return SSM_ERR_INVALID_ARGUMENT;
    return strides_fit(v->sb, v->sh, v->sl) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

int check_group_view(const ssm_group_view* v, int dtype, bool output, const ssm_sequences* q, int64_t N, int64_t G) {
    if (!v->data) return SSM_ERR_INVALID_ARGUMENT;
    if (!aligned(v->data, type_bytes(dtype)) || v->sb < 0 || v->sg < 0 || v->sn < 0 || v->sl < 0)
        return SSM_ERR_INVALID_ARGUMENT;
    if (output && ((v->sb == 0 && q->Bsz > 1) || (v->sg == 0 && G > 1) || (v->sn == 0 && N > 1) ||
                   (v->sl == 0 && q->L > 1)))
        return SSM_ERR_INVALID_ARGUMENT;
    return v->sg < ((int64_t)1 << 40) && strides_fit(v->sb, v->sn, v->sl) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

View3 view_of(const ssm_view* v) {
    View3 r;
    if (v) r.data = v->data, r.sb = v->sb, r.sh = v->sh, r.sl = v->sl;
    return r;
}
View4 view_of(const ssm_group_view& v) {
    View4 r;
    r.data = v.data, r.sb = v.sb, r.sg = v.sg, r.sn = v.sn, r.sl = v.sl;
    return r;
}

#define SSM_TRY(expr)                   \
    do {                                \
        const int rc_ = (expr);         \
        if (rc_ != SSM_OK) return rc_;  \
    } while (0)

int check_conv(int dtype, const ssm_sequences* seq, int64_t H, int64_t width, int silu, const ssm_view* u,
               const float* weight, const float* bias, const void* state_in, bool slots_allowed, ConvArgs* a) {
    if (!type_known(dtype) || H < 1 || width < 1) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_sequences(seq, H, slots_allowed, &a->q));
    if (width > kMaxWidth) return SSM_ERR_UNSUPPORTED;
    SSM_TRY(check_view(u, dtype, true, false, seq, H));
    if (!weight || (width == 1 && state_in)) return SSM_ERR_INVALID_ARGUMENT;
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(state_in, type_bytes(dtype)))
        return SSM_ERR_INVALID_ARGUMENT;
    if (!conv_fits(a->q, H)) return SSM_ERR_UNSUPPORTED;
    a->H = H;
    a->width = (int)width;
    a->silu = silu;
    a->u = view_of(u);
    a->weight = weight;
    a->bias = bias;
    a->state_in = state_in;
    a->state_out = nullptr;
    return SSM_OK;
}

int check_scan(const ssm_sequences* seq, const ssm_selective* p, bool slots_allowed, ScanArgs* a) {
    if (!p || !type_known(p->dtype) || p->H < 1) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_sequences(seq, p->H, slots_allowed, &a->q));
    SSM_TRY(check_scan_sizes(p->H, p->N, p->G));
    SSM_TRY(check_view(&p->u, p->dtype, true, false, seq, p->H));
    SSM_TRY(check_view(&p->delta, p->dtype, true, false, seq, p->H));
    SSM_TRY(check_view(&p->z, p->dtype, false, false, seq, p->H));
    SSM_TRY(check_group_view(&p->B, p->dtype, false, seq, p->N, p->G));
    SSM_TRY(check_group_view(&p->C, p->dtype, false, seq, p->N, p->G));
    const float* f[] = {p->A, p->D, p->delta_bias, p->x_in};
    for (const float* v : f)
        if (!aligned(v, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (!p->A) return SSM_ERR_INVALID_ARGUMENT;
    if (!scan_fits(a->q, p->H, p->N, p->G)) return SSM_ERR_UNSUPPORTED;
    a->Bsz = seq->Bsz;
    a->H = p->H;
    a->N = p->N;
    a->G = p->G;
    a->softplus = p->softplus;
    a->u = view_of(&p->u);
    a->delta = view_of(&p->delta);
    a->z = view_of(&p->z);
    a->B = view_of(p->B);
    a->C = view_of(p->C);
    a->A = p->A;
    a->D = p->D;
    a->delta_bias = p->delta_bias;
    a->x_in = p->x_in;
    a->x_out = nullptr;
    a->saved = nullptr;
    return SSM_OK;
}

size_t saved_bytes_of(const Seqs& q, int64_t H, int64_t N) {
    return (size_t)saved_rows(q.S, q.L, q.offsets != nullptr) * H * padded_states(N) * sizeof(float);
}

}  // namespace

extern "C" {

int ssm_selective_bytes(int op, int64_t Bsz, int64_t H, int64_t N, int64_t G, int64_t L, int64_t S, int packed,
                        size_t* bytes) {
    if (!bytes) return SSM_ERR_INVALID_ARGUMENT;
    if (op < SSM_OP_SELECTIVE_SCAN || op > SSM_OP_CAUSAL_CONV_BACKWARD) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_sizes(Bsz, H, L, S, packed != 0));
    const Seqs q = sequences_of(L, S, packed != 0);
    if (op == SSM_OP_CAUSAL_CONV_BACKWARD) {
        if (N < 1) return SSM_ERR_INVALID_ARGUMENT;
        if (N > kMaxWidth || !conv_fits(q, H)) return SSM_ERR_UNSUPPORTED;
        *bytes = conv_grad_workspace_bytes(q, H, (int)N);
        return SSM_OK;
    }
    SSM_TRY(check_scan_sizes(H, N, G));
    if (!scan_fits(q, H, N, G)) return SSM_ERR_UNSUPPORTED;
    if (op == SSM_OP_SELECTIVE_SCAN) {
        *bytes = scan_workspace_bytes(q, H, N, G);
    } else if (op == SSM_OP_SELECTIVE_SAVED) {
        *bytes = saved_bytes_of(q, H, N);
    } else {
        if (!scan_grad_fits(q, Bsz, H, N, G)) return SSM_ERR_UNSUPPORTED;
        *bytes = scan_grad_workspace_bytes(q, Bsz, H, N, G);
    }
    return SSM_OK;
}

int ssm_causal_conv(int dtype, const ssm_sequences* seq, int64_t H, int64_t width, int silu, const ssm_view* u,
                    const float* weight, const float* bias, const void* state_in, void* state_out,
                    const ssm_view* y, void* stream) {
    ConvArgs a;
    SSM_TRY(check_conv(dtype, seq, H, width, silu, u, weight, bias, state_in, true, &a));
    SSM_TRY(check_view(y, dtype, true, true, seq, H));
    if (!aligned(state_out, type_bytes(dtype)) || (width == 1 && state_out)) return SSM_ERR_INVALID_ARGUMENT;
    a.y = view_of(y);
    a.state_out = state_out;
    return device_status(launch_causal_conv(dtype, a, (hipStream_t)stream));
}

int ssm_causal_conv_backward(int dtype, const ssm_sequences* seq, int64_t H, int64_t width, int silu,
                             const ssm_view* u, const float* weight, const float* bias, const void* state_in,
                             const ssm_view* dy, const float* dstate_out, const ssm_view* du, float* dweight,
                             float* dbias, float* dstate_in, void* ws, size_t ws_bytes, void* stream) {
    ConvGradArgs g;
    SSM_TRY(check_conv(dtype, seq, H, width, silu, u, weight, bias, state_in, false, &g.f));
    SSM_TRY(check_view(dy, dtype, true, false, seq, H));
    SSM_TRY(check_view(du, dtype, true, true, seq, H));
    const float* f[] = {dstate_out, dweight, dbias, dstate_in};
    for (const float* v : f)
        if (!aligned(v, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (width == 1 && (dstate_out || dstate_in)) return SSM_ERR_INVALID_ARGUMENT;
    if (!aligned(ws, 256)) return SSM_ERR_INVALID_ARGUMENT;
    if ((dweight || dbias) && (!ws || ws_bytes < conv_grad_workspace_bytes(g.f.q, H, (int)width)))
        return SSM_ERR_WORKSPACE;
    g.dy = view_of(dy);
    g.du = view_of(du);
    g.dweight = dweight;
    g.dbias = dbias;
    g.dstate_out = dstate_out;
    g.dstate_in = dstate_in;
    return device_status(launch_causal_conv_backward(dtype, g, ws, (hipStream_t)stream));
}

int ssm_causal_conv_step(int dtype, int64_t Bsz, int64_t H, int64_t width, int silu, const void* u, int64_t u_stride,
                         const float* weight, const float* bias, void* state, const int32_t* slots,
                         int64_t n_slots, void* y, int64_t y_stride, void* stream) {
    if (!type_known(dtype) || Bsz < 1 || H < 1 || width < 1) return SSM_ERR_INVALID_ARGUMENT;
    if (width > kMaxWidth || Bsz >= kMaxDim || H >= kMaxDim || Bsz * H >= kMaxDim) return SSM_ERR_UNSUPPORTED;
    if (!u || !weight || !y || (width > 1) != (state != nullptr) || u_stride < 0 || y_stride < 0 ||
        (y_stride == 0 && Bsz > 1) || (slots && n_slots < 1))
        return SSM_ERR_INVALID_ARGUMENT;
    const size_t e = type_bytes(dtype);
    if (!aligned(u, e) || !aligned(y, e) || !aligned(state, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(slots, 4))
        return SSM_ERR_INVALID_ARGUMENT;
    if (u_stride >= ((int64_t)1 << 32) || y_stride >= ((int64_t)1 << 32) ||
        (slots && n_slots > ((int64_t)1 << 40) / H))
        return SSM_ERR_UNSUPPORTED;
    ConvStepArgs a;
    a.Bsz = Bsz;
    a.H = H;
    a.width = (int)width;
    a.silu = silu;
    a.slots = slots;
    a.n_slots = slots ? n_slots : Bsz;
    a.u = u;
    a.y = y;
    a.u_row = u_stride;
    a.y_row = y_stride;
    a.weight = weight;
    a.bias = bias;
    a.state = state;
    return device_status(launch_causal_conv_step(dtype, a, (hipStream_t)stream));
}

int ssm_selective_scan(const ssm_sequences* seq, const ssm_selective* p, const ssm_view* y, float* x_out, void* saved,
                       size_t saved_bytes, void* ws, size_t ws_bytes, void* stream) {
    ScanArgs a;
    SSM_TRY(check_scan(seq, p, true, &a));
    SSM_TRY(check_view(y, p->dtype, !saved && !x_out, true, seq, p->H));
    if (!aligned(x_out, 4) || !aligned(saved, 256) || !aligned(ws, 256)) return SSM_ERR_INVALID_ARGUMENT;
    if (saved && seq->slots) return SSM_ERR_INVALID_ARGUMENT;
    if (saved && saved_bytes < saved_bytes_of(a.q, a.H, a.N)) return SSM_ERR_WORKSPACE;
    const size_t need = scan_workspace_bytes(a.q, a.H, a.N, a.G);
    if (need && (!ws || ws_bytes < need)) return SSM_ERR_WORKSPACE;
    a.y = view_of(y);
    a.x_out = x_out;
    a.saved = (float*)saved;
    return device_status(launch_scan(p->dtype, a, ws, (hipStream_t)stream));
}

int ssm_selective_scan_backward(const ssm_sequences* seq, const ssm_selective* p, const void* saved,
                                size_t saved_bytes, const ssm_view* dy, const float* dx_out,
                                const ssm_selective_grads* grads, void* ws, size_t ws_bytes, void* stream) {
    ScanGradArgs g;
    SSM_TRY(check_scan(seq, p, false, &g.f));
    if (!grads || !saved || !aligned(saved, 256) || !aligned(ws, 256)) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_view(dy, p->dtype, true, false, seq, p->H));
    SSM_TRY(check_view(&grads->du, p->dtype, true, true, seq, p->H));
    SSM_TRY(check_view(&grads->ddelta, p->dtype, true, true, seq, p->H));
    SSM_TRY(check_view(&grads->dz, p->dtype, p->z.data != nullptr, true, seq, p->H));
    if (!p->z.data && grads->dz.data) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_group_view(&grads->dB, p->dtype, true, seq, p->N, p->G));
    SSM_TRY(check_group_view(&grads->dC, p->dtype, true, seq, p->N, p->G));
    const float* f[] = {dx_out, grads->dA, grads->dD, grads->ddelta_bias, grads->dx_in};
    for (const float* v : f)
        if (!aligned(v, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (!grads->dA) return SSM_ERR_INVALID_ARGUMENT;
    if (!scan_grad_fits(g.f.q, seq->Bsz, p->H, p->N, p->G)) return SSM_ERR_UNSUPPORTED;
    if (saved_bytes < saved_bytes_of(g.f.q, p->H, p->N)) return SSM_ERR_WORKSPACE;
    if (!ws || ws_bytes < scan_grad_workspace_bytes(g.f.q, seq->Bsz, p->H, p->N, p->G)) return SSM_ERR_WORKSPACE;
    g.saved = (const float*)saved;
    g.dy = view_of(dy);
    g.du = view_of(&grads->du);
    g.ddelta = view_of(&grads->ddelta);
    g.dz = view_of(&grads->dz);
    g.dB = view_of(grads->dB);
    g.dC = view_of(grads->dC);
    g.dA = grads->dA;
    g.dD = grads->dD;
    g.ddelta_bias = grads->ddelta_bias;
    g.dx_out = dx_out;
    g.dx_in = grads->dx_in;
    return device_status(launch_scan_backward(p->dtype, g, ws, (hipStream_t)stream));
}

int ssm_selective_step(const ssm_selective_token* p, void* stream) {
    if (!p || !type_known(p->dtype) || p->Bsz < 1 || p->H < 1) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_scan_sizes(p->H, p->N, p->G));
    if (p->Bsz >= kMaxDim || p->H >= kMaxDim || p->Bsz * p->H >= kMaxDim ||
        !grid_fits(p->Bsz * ((p->H + 63) / 64), 256))
        return SSM_ERR_UNSUPPORTED;
    if (!p->u || !p->delta || !p->B || !p->C || !p->y || !p->A || !p->x || (p->slots && p->n_slots < 1))
        return SSM_ERR_INVALID_ARGUMENT;
    const size_t e = type_bytes(p->dtype);
    const void* acts[] = {p->u, p->delta, p->z, p->B, p->C, p->y};
    for (const void* v : acts)
        if (!aligned(v, e)) return SSM_ERR_INVALID_ARGUMENT;
    const void* words[] = {p->slots, p->A, p->D, p->delta_bias, p->x};
    for (const void* v : words)
        if (!aligned(v, 4)) return SSM_ERR_INVALID_ARGUMENT;
    const int64_t strides[] = {p->u_stride, p->delta_stride, p->z_stride, p->y_stride, p->B_stride,
                               p->B_group,  p->B_state,      p->C_stride, p->C_group,  p->C_state};
    for (int64_t s : strides)
        if (s < 0) return SSM_ERR_INVALID_ARGUMENT;
    if (p->y_stride == 0 && p->Bsz > 1) return SSM_ERR_INVALID_ARGUMENT;
    for (int64_t s : strides)
        if (s >= ((int64_t)1 << 32)) return SSM_ERR_UNSUPPORTED;
    if (p->slots && p->n_slots > ((int64_t)1 << 40) / p->H) return SSM_ERR_UNSUPPORTED;
    StepArgs a;
    a.Bsz = p->Bsz;
    a.H = p->H;
    a.N = p->N;
    a.G = p->G;
    a.softplus = p->softplus;
    a.slots = p->slots;
    a.n_slots = p->slots ? p->n_slots : p->Bsz;
    a.u = p->u, a.delta = p->delta, a.z = p->z, a.B = p->B, a.C = p->C, a.y = p->y;
    a.u_row = p->u_stride, a.delta_row = p->delta_stride, a.z_row = p->z_stride, a.y_row = p->y_stride;
    a.B_row = p->B_stride, a.B_group = p->B_group, a.B_state = p->B_state;
    a.C_row = p->C_stride, a.C_group = p->C_group, a.C_state = p->C_state;
    a.A = p->A, a.D = p->D, a.delta_bias = p->delta_bias, a.x = p->x;
    return device_status(launch_selective_step(p->dtype, a, (hipStream_t)stream));
}

}  // extern "C"

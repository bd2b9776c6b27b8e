// C ABI entry points of layer norm: argument checks and launches.
#include "checks.hpp"
#include "norm.hpp"

using namespace ssm;

namespace {

int check_norm_sizes(int64_t Bsz, int64_t H, int64_t L, int64_t G) {
    SSM_TRY(check_sizes(Bsz, H, L, Bsz, false));
    return G < 1 || H % G != 0 ? SSM_ERR_INVALID_ARGUMENT : SSM_OK;
}

int check_norm(const ssm_norm* p, ssm_sequences* q, NormArgs* a) {
    if (!p || !type_known(p->dtype) || p->gate < SSM_GATE_NONE || p->gate > SSM_GATE_AFTER) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_norm_sizes(p->Bsz, p->H, p->L, p->G));
    q->Bsz = p->Bsz, q->L = p->L;
    SSM_TRY(check_view(&p->u, p->dtype, true, false, q, p->H));
    SSM_TRY(check_view(&p->z, p->dtype, p->gate != SSM_GATE_NONE, false, q, p->H));
    if ((p->gate == SSM_GATE_NONE && p->z.data) || !aligned(p->weight, 4) || !aligned(p->bias, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (!(p->eps >= 0.0f) || !(p->eps < INFINITY)) return SSM_ERR_INVALID_ARGUMENT;
    a->Bsz = p->Bsz, a->H = p->H, a->L = p->L, a->G = p->G;
    a->rms = p->rms, a->gate = p->gate;
    a->eps = p->eps;
    a->u = view_of(&p->u), a->z = view_of(&p->z);
    a->weight = p->weight, a->bias = p->bias;
    return SSM_OK;
}

size_t backward_bytes(int64_t Bsz, int64_t H, int64_t L, int64_t G) {
    return (size_t)(2 * norm_part_rows(Bsz, L, H / G, G)) * H * sizeof(float);
}

}  // namespace

extern "C" {

int ssm_layer_norm_bytes(int64_t Bsz, int64_t H, int64_t L, int64_t G, size_t* bytes) {
    if (!bytes) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_norm_sizes(Bsz, H, L, G));
    if (!norm_grad_may_fit(Bsz, L, H / G, G)) return SSM_ERR_UNSUPPORTED;
    *bytes = backward_bytes(Bsz, H, L, G);
    return SSM_OK;
}

int ssm_layer_norm(const ssm_norm* p, const ssm_view* y, void* stream) {
    NormArgs a;
    ssm_sequences q = {};
    SSM_TRY(check_norm(p, &q, &a));
    SSM_TRY(check_view(y, p->dtype, true, true, &q, p->H));
    a.y = view_of(y);
    if (!norm_fits(a)) return SSM_ERR_UNSUPPORTED;
    return device_status(launch_norm(p->dtype, a, (hipStream_t)stream));
}

int ssm_layer_norm_backward(const ssm_norm* p, const ssm_view* dy, const ssm_view* du, const ssm_view* dz, float* dweight,
                            float* dbias, void* ws, size_t ws_bytes, void* stream) {
    NormGradArgs g;
    ssm_sequences q = {};
    SSM_TRY(check_norm(p, &q, &g.f));
    SSM_TRY(check_view(dy, p->dtype, true, false, &q, p->H));
    SSM_TRY(check_view(du, p->dtype, true, true, &q, p->H));
    SSM_TRY(check_view(dz, p->dtype, p->gate != SSM_GATE_NONE, true, &q, p->H));
    if ((p->gate == SSM_GATE_NONE && dz && dz->data) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(ws, 256))
        return SSM_ERR_INVALID_ARGUMENT;
    g.dy = view_of(dy), g.du = view_of(du), g.dz = view_of(dz);
    if (!norm_fits(g)) return SSM_ERR_UNSUPPORTED;
    const bool sums = dweight || dbias;
    if (sums && (!ws || ws_bytes < backward_bytes(p->Bsz, p->H, p->L, p->G))) return SSM_ERR_WORKSPACE;
    g.dweight = dweight, g.dbias = dbias;
    g.parts = sums ? (float*)ws : nullptr;
    g.rows = 0;
    return device_status(launch_norm_backward(p->dtype, g, (hipStream_t)stream));
}

}  // extern "C"

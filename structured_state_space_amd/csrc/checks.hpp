// Argument checks of the C ABI that the operators on views and sequences share
// (host code).
#pragma once

#include "selective.hpp"

namespace ssm {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
// a thread's distance from its workgroup's first channel (or state) and step is
// 32 bits wide in bytes: up to 67 channels or 64 states, and 32 steps, of 4 bytes
constexpr int64_t kMaxStride = (int64_t)1 << 23;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool type_known(int dtype) { return dtype == SSM_F32 || dtype == SSM_BF16 || dtype == SSM_F16; }
inline size_t type_bytes(int dtype) { return dtype == SSM_F32 ? 4 : 2; }
inline int device_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_DEVICE; }

// sizes of a call on whole sequences
inline int check_sizes(int64_t Bsz, int64_t H, int64_t L, int64_t S, bool packed) {
    if (Bsz < 1 || H < 1 || L < 1 || S < 1 || (packed ? Bsz != 1 : S != Bsz)) return SSM_ERR_INVALID_ARGUMENT;
    if (Bsz >= kMaxDim || H >= kMaxDim || L >= kMaxDim - 64 || S >= kMaxDim - 64 || Bsz * H >= kMaxDim ||
        S * H >= kMaxDim || Bsz * H > ((int64_t)1 << 40) / L)
        return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

inline int check_sequences(const ssm_sequences* q, int64_t H, bool slots_allowed, Seqs* out) {
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

inline Seqs sequences_of(int64_t L, int64_t S, bool packed) {
    Seqs q;
    q.S = S;
    q.L = L;
    q.offsets = packed ? reinterpret_cast<const int32_t*>(16) : nullptr;  // only tested for null by the size rules
    return q;
}

// an output's dimensions of more than one element must not be broadcast
inline bool strides_fit(int64_t sb, int64_t sh, int64_t sl) {
    return sb < ((int64_t)1 << 40) && sh < kMaxStride && sl < kMaxStride;
}

inline int check_view(const ssm_view* v, int dtype, bool required, bool output, const ssm_sequences* q, int64_t H) {
    if (!v || !v->data) return required ? SSM_ERR_INVALID_ARGUMENT : SSM_OK;
    if (!aligned(v->data, type_bytes(dtype)) || v->sb < 0 || v->sh < 0 || v->sl < 0) return SSM_ERR_INVALID_ARGUMENT;
    if (output && ((v->sb == 0 && q->Bsz > 1) || (v->sh == 0 && H > 1) || (v->sl == 0 && q->L > 1)))
        return SSM_ERR_INVALID_ARGUMENT;
    return strides_fit(v->sb, v->sh, v->sl) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

inline int check_group_view(const ssm_group_view* v, int dtype, bool output, const ssm_sequences* q, int64_t N, int64_t G) {
    if (!v->data) return SSM_ERR_INVALID_ARGUMENT;
    if (!aligned(v->data, type_bytes(dtype)) || v->sb < 0 || v->sg < 0 || v->sn < 0 || v->sl < 0)
        return SSM_ERR_INVALID_ARGUMENT;
    if (output && ((v->sb == 0 && q->Bsz > 1) || (v->sg == 0 && G > 1) || (v->sn == 0 && N > 1) ||
                   (v->sl == 0 && q->L > 1)))
        return SSM_ERR_INVALID_ARGUMENT;
    return v->sg < ((int64_t)1 << 40) && strides_fit(v->sb, v->sn, v->sl) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

inline View3 view_of(const ssm_view* v) {
    View3 r;
    if (v) r.data = v->data, r.sb = v->sb, r.sh = v->sh, r.sl = v->sl;
    return r;
}
inline View4 view_of(const ssm_group_view& v) {
    View4 r;
    r.data = v.data, r.sb = v.sb, r.sg = v.sg, r.sn = v.sn, r.sl = v.sl;
    return r;
}

#define SSM_TRY(expr)                   \
    do {                                \
        const int rc_ = (expr);         \
        if (rc_ != SSM_OK) return rc_;  \
    } while (0)

}  // namespace ssm

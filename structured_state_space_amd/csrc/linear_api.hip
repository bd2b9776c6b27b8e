// C ABI entry points of linear attention: argument checks, sizes, the split into
// segments and the order of the launches.
#include "checks.hpp"
#include "linear.hpp"

namespace ssm {
template <class T, bool REVERSE>
hipError_t launch_walk(const WalkArgs& a, hipStream_t s);
template <class T>
hipError_t launch_pairs(const PairArgs& a, hipStream_t s);
extern template hipError_t launch_walk<float, false>(const WalkArgs&, hipStream_t);
extern template hipError_t launch_walk<float, true>(const WalkArgs&, hipStream_t);
extern template hipError_t launch_walk<bf16, false>(const WalkArgs&, hipStream_t);
extern template hipError_t launch_walk<bf16, true>(const WalkArgs&, hipStream_t);
extern template hipError_t launch_walk<f16, false>(const WalkArgs&, hipStream_t);
extern template hipError_t launch_walk<f16, true>(const WalkArgs&, hipStream_t);
extern template hipError_t launch_pairs<float>(const PairArgs&, hipStream_t);
extern template hipError_t launch_pairs<bf16>(const PairArgs&, hipStream_t);
extern template hipError_t launch_pairs<f16>(const PairArgs&, hipStream_t);
bool linear_step_fits(int64_t Bsz, int64_t H, int64_t P);
hipError_t launch_linear_step(int dtype, const LinearStepArgs& a, hipStream_t s);
}  // namespace ssm

using namespace ssm;

namespace {

struct Sizes {
    int64_t Bsz, H, G, N, P;
    int dtype;
};
int chunk_of(int dtype) { return dtype == SSM_F32 ? kChunk<float> : kChunk<bf16>; }
int64_t value_blocks(int64_t P) { return (P + 63) / 64; }
size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Steps of a segment, whole chunks.  A walk has a workgroup per sequence, head and 64
// values; where those leave many of the compute units idle, sequences are cut, for one more
// launch over nearly all of the steps, which finds every segment's end state.  Forwards,
// 128 keys, 64 values, bf16, cut and not cut: 32 workgroups of 4096 steps 73 and 237 us, 96 146
// and 238, 128 of 8192 281 and 467, 200 of 4096 252 and 236; 160 in float32 514 and 591.
// Cut into about 512 workgroups: 32 heads of 16384 steps 190 us, into 256 211, 1024 236; of four
// chunks or more, since every segment starts with its state and the first loads' latency.
int64_t segment_steps(const Seqs& q, const Sizes& z) {
    const int64_t Q = chunk_of(z.dtype), wgs = (q.offsets ? 1 : q.S) * z.H * value_blocks(z.P);
    int64_t steps = q.L;
    if (wgs <= 160) {
        const int64_t cuts = (512 + wgs - 1) / wgs;
        steps = (q.L + cuts - 1) / cuts;
        if (steps < 4 * Q) steps = 4 * Q;
    }
    steps = (steps + Q - 1) / Q * Q;
    return steps < ((int64_t)1 << 30) ? steps : (int64_t)1 << 30;
}
size_t walk_bytes(const Seqs& q, const Sizes& z) {
    const int64_t seg = segment_steps(q, z);
    if (seg >= q.L) return 0;
    const int64_t items = item_count(q, seg);
    return rounded((size_t)(items * z.H) * z.N * z.P * sizeof(float)) + rounded((size_t)(items * z.H) * sizeof(float));
}
size_t saved_bytes(const Seqs& q, const Sizes& z) {
    return (size_t)(linear_rows(q.S, q.L, q.offsets != nullptr, chunk_of(z.dtype)) * z.H) * padded_keys(z.N) *
           padded_values(z.P) * sizeof(float);
}
// Workgroups that share a group's heads in the pairs' kernel, and their heads: as many as the
// compute units take at once.  More add partial sums and fewer heads to each pipeline: forwards
// and backwards at 4 x 2048 steps, 64 heads, one group, bf16, 551 us with twice and 563 with four times as
// many, 533 so; 80 heads in eight groups over 1024 steps 179, 193 and 158.  Small tiles of float32
// have two workgroups to a unit: 2 x 2048 steps, 32 heads, 255 us, with half 268, with twice 262.
int64_t head_blocks(const Seqs& q, const Sizes& z, int* heads) {
    const int64_t items = item_count(q, chunk_of(z.dtype)), Hg = z.H / z.G;
    const int64_t all = z.dtype == SSM_F32 && z.N <= 64 ? 512 : 256;
    int64_t blocks = (all + items * z.G - 1) / (items * z.G);
    if (blocks > Hg) blocks = Hg;
    if (blocks > 8) blocks = 8;
    const int64_t each = (Hg + blocks - 1) / blocks;
    *heads = (int)each;
    return (Hg + each - 1) / each;
}
struct GradLayout {
    size_t ahead, parts, skips, walk, bytes;
};
GradLayout grad_layout(const Seqs& q, const Sizes& z) {
    GradLayout l;
    int heads;
    const int64_t blocks = head_blocks(q, z, &heads);
    l.ahead = 0;
    l.parts = l.ahead + rounded(saved_bytes(q, z));
    l.skips = l.parts + (blocks > 1 ? rounded((size_t)(blocks * 2 * z.Bsz) * z.G * q.L * z.N * sizeof(float)) : 0);
    l.walk = l.skips + rounded((size_t)(item_count(q, chunk_of(z.dtype)) * z.H) * sizeof(float));
    l.bytes = l.walk + walk_bytes(q, z);
    return l;
}

int check_linear_sizes(int64_t H, int64_t N, int64_t P, int64_t G) {
    if (H < 1 || N < 1 || P < 1 || G < 1 || H % G != 0) return SSM_ERR_INVALID_ARGUMENT;
    return N > kMaxKeys || P > kMaxValues ? SSM_ERR_UNSUPPORTED : SSM_OK;
}
bool grids_fit(const Seqs& q, const Sizes& z) {
    const int64_t chunks = item_count(q, chunk_of(z.dtype));
    return grid_fits(item_count(q, segment_steps(q, z)) * z.H * value_blocks(z.P), 512) &&
           grid_fits(chunks * z.G * 8 + z.H, 512) &&
           chunks * z.H < ((int64_t)1 << 40) / (padded_keys(z.N) * padded_values(z.P));
}

int check_linear(const ssm_sequences* seq, const ssm_linear* p, bool slots_allowed, LinearArgs* a, Sizes* z) {
    if (!p || !type_known(p->dtype)) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_linear_sizes(p->H, p->N, p->P, p->G));
    SSM_TRY(check_sequences(seq, p->H, slots_allowed, &a->q));
    SSM_TRY(check_group_view(&p->q, p->dtype, false, seq, p->N, p->G));
    SSM_TRY(check_group_view(&p->k, p->dtype, false, seq, p->N, p->G));
    SSM_TRY(check_group_view(&p->v, p->dtype, false, seq, p->P, p->H));
    SSM_TRY(check_view(&p->g, SSM_F32, true, false, seq, p->H));
    SSM_TRY(check_view(&p->beta, SSM_F32, false, false, seq, p->H));
    if (!aligned(p->D, 4) || !aligned(p->x_in, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (!(p->scale - p->scale == 0.0f)) return SSM_ERR_INVALID_ARGUMENT;
    *z = Sizes{seq->Bsz, p->H, p->G, p->N, p->P, p->dtype};
    if (!grids_fit(a->q, *z)) return SSM_ERR_UNSUPPORTED;
    a->Bsz = seq->Bsz;
    a->H = p->H;
    a->G = p->G;
    a->N = p->N;
    a->P = p->P;
    a->scale = p->scale;
    a->qv = view_of(p->q);
    a->k = view_of(p->k);
    a->v = view_of(p->v);
    a->g = view_of(&p->g);
    a->beta = view_of(&p->beta);
    a->D = p->D;
    a->x_in = p->x_in;
    return SSM_OK;
}

template <bool REVERSE>
hipError_t walk(const LinearArgs& a, const Sizes& z, const View4& value, const View4& result, const float* x_in,
                float* x_out, float* saved, void* ws, hipStream_t s) {
    WalkArgs w;
    w.q = a.q;
    w.H = a.H, w.G = a.G, w.N = a.N, w.P = a.P;
    const int64_t size = type_bytes(z.dtype);
    w.key = source_of(REVERSE ? a.qv : a.k, a.N, size), w.query = source_of(REVERSE ? a.k : a.qv, a.N, size);
    w.value = source_of(value, a.P, size), w.result = result;
    w.fast = w.key.lay == kByColumn && w.query.lay == kByColumn && w.value.lay == kByColumn && (!result.data || result.sn == 1);
    w.g = a.g, w.beta = a.beta;
    w.scale = a.scale;
    w.D = a.D;
    w.x_in = x_in, w.x_out = x_out, w.saved = saved;
    w.segment = segment_steps(a.q, z);
    w.items = item_count(a.q, w.segment);
    w.seg_x = (float*)ws;
    w.seg_decay = ws ? (float*)((char*)ws + rounded((size_t)(w.items * a.H) * a.N * a.P * sizeof(float))) : nullptr;
    if (z.dtype == SSM_F32) return launch_walk<float, REVERSE>(w, s);
    if (z.dtype == SSM_BF16) return launch_walk<bf16, REVERSE>(w, s);
    return launch_walk<f16, REVERSE>(w, s);
}

}  // namespace

extern "C" {

int ssm_linear_bytes(int op, int dtype, int64_t Bsz, int64_t H, int64_t N, int64_t P, int64_t G, int64_t L, int64_t S,
                     int packed, size_t* bytes) {
    if (!bytes || !type_known(dtype)) return SSM_ERR_INVALID_ARGUMENT;
    if (op < SSM_OP_LINEAR_ATTENTION || op > SSM_OP_LINEAR_SAVED) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_linear_sizes(H, N, P, G));
    SSM_TRY(check_sizes(Bsz, H, L, S, packed != 0));
    const Seqs q = sequences_of(L, S, packed != 0);
    const Sizes z{Bsz, H, G, N, P, dtype};
    if (!grids_fit(q, z)) return SSM_ERR_UNSUPPORTED;
    if (op == SSM_OP_LINEAR_ATTENTION) *bytes = walk_bytes(q, z);
    else if (op == SSM_OP_LINEAR_SAVED) *bytes = saved_bytes(q, z);
    else *bytes = grad_layout(q, z).bytes;
    return SSM_OK;
}

int ssm_linear_attention(const ssm_sequences* seq, const ssm_linear* p, const ssm_group_view* y, float* x_out,
                         void* saved, size_t saved_size, void* ws, size_t ws_bytes, void* stream) {
    LinearArgs a;
    Sizes z;
    SSM_TRY(check_linear(seq, p, true, &a, &z));
    if (!y || !y->data) {
        if (!saved && !x_out) return SSM_ERR_INVALID_ARGUMENT;
    } else {
        SSM_TRY(check_group_view(y, p->dtype, true, seq, p->P, p->H));
    }
    if (!aligned(x_out, 4) || !aligned(saved, 256) || !aligned(ws, 256)) return SSM_ERR_INVALID_ARGUMENT;
    if (saved && seq->slots) return SSM_ERR_INVALID_ARGUMENT;
    if (saved && saved_size < saved_bytes(a.q, z)) return SSM_ERR_WORKSPACE;
    const size_t need = walk_bytes(a.q, z);
    if (need && (!ws || ws_bytes < need)) return SSM_ERR_WORKSPACE;
    return device_status(walk<false>(a, z, a.v, y ? view_of(*y) : View4(), a.x_in, x_out, (float*)saved, ws,
                                     (hipStream_t)stream));
}

int ssm_linear_attention_backward(const ssm_sequences* seq, const ssm_linear* p, const void* saved, size_t saved_size,
                                  const ssm_group_view* dy, const float* dx_out, const ssm_linear_grads* grads, void* ws,
                                  size_t ws_bytes, void* stream) {
    LinearArgs a;
    Sizes z;
    SSM_TRY(check_linear(seq, p, false, &a, &z));
    if (!dy || !grads || !saved || !aligned(saved, 256) || !aligned(ws, 256)) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_group_view(dy, p->dtype, false, seq, p->P, p->H));
    SSM_TRY(check_group_view(&grads->dq, p->dtype, true, seq, p->N, p->G));
    SSM_TRY(check_group_view(&grads->dk, p->dtype, true, seq, p->N, p->G));
    SSM_TRY(check_group_view(&grads->dv, p->dtype, true, seq, p->P, p->H));
    SSM_TRY(check_view(&grads->dg, SSM_F32, true, true, seq, p->H));
    SSM_TRY(check_view(&grads->dbeta, SSM_F32, false, true, seq, p->H));
    if ((!p->beta.data && grads->dbeta.data) || (!p->D && grads->dD)) return SSM_ERR_INVALID_ARGUMENT;
    if (!aligned(grads->dD, 4) || !aligned(grads->dx_in, 4) || !aligned(dx_out, 4)) return SSM_ERR_INVALID_ARGUMENT;
    if (saved_size < saved_bytes(a.q, z)) return SSM_ERR_WORKSPACE;
    const GradLayout l = grad_layout(a.q, z);
    if (!ws || ws_bytes < l.bytes) return SSM_ERR_WORKSPACE;
    char* base = (char*)ws;
    float* ahead = (float*)(base + l.ahead);
    const hipError_t e = walk<true>(a, z, view_of(*dy), view_of(grads->dv), dx_out, grads->dx_in, ahead, base + l.walk,
                                    (hipStream_t)stream);
    if (e != hipSuccess) return device_status(e);
    PairArgs r;
    r.q = a.q;
    r.Bsz = a.Bsz, r.H = a.H, r.G = a.G, r.N = a.N, r.P = a.P;
    r.scale = a.scale;
    const int64_t size = type_bytes(z.dtype);
    r.qv = source_of(a.qv, a.N, size), r.k = source_of(a.k, a.N, size);
    r.v = source_of(a.v, a.P, size), r.dy = source_of(view_of(*dy), a.P, size);
    r.dq = view_of(grads->dq), r.dk = view_of(grads->dk);
    r.fast = r.qv.lay == kByColumn && r.k.lay == kByColumn && r.v.lay == kByColumn && r.dy.lay == kByColumn;
    r.g = a.g, r.beta = a.beta, r.dg = view_of(&grads->dg), r.dbeta = view_of(&grads->dbeta);
    r.states = (const float*)saved, r.ahead = ahead;
    r.blocks = (int)head_blocks(a.q, z, &r.heads);
    r.items = item_count(a.q, chunk_of(z.dtype));
    r.parts = (float*)(base + l.parts);
    r.skips = grads->dD ? (float*)(base + l.skips) : nullptr;
    r.dD = grads->dD;
    const hipStream_t s = (hipStream_t)stream;
    return device_status(z.dtype == SSM_F32 ? launch_pairs<float>(r, s)
                         : z.dtype == SSM_BF16 ? launch_pairs<bf16>(r, s) : launch_pairs<f16>(r, s));
}

int ssm_linear_attention_step(const ssm_linear_token* p, void* stream) {
    if (!p || !type_known(p->dtype) || p->Bsz < 1) return SSM_ERR_INVALID_ARGUMENT;
    SSM_TRY(check_linear_sizes(p->H, p->N, p->P, p->G));
    if (p->Bsz >= kMaxDim || p->H >= kMaxDim || p->Bsz * p->H >= kMaxDim || !linear_step_fits(p->Bsz, p->H, p->P))
        return SSM_ERR_UNSUPPORTED;
    if (!p->q || !p->k || !p->v || !p->g || !p->y || !p->x || (p->slots && p->n_slots < 1))
        return SSM_ERR_INVALID_ARGUMENT;
    if (!(p->scale - p->scale == 0.0f)) return SSM_ERR_INVALID_ARGUMENT;
    const size_t e = type_bytes(p->dtype);
    const void* acts[] = {p->q, p->k, p->v, p->y};
    for (const void* v : acts)
        if (!aligned(v, e)) return SSM_ERR_INVALID_ARGUMENT;
    const void* words[] = {p->slots, p->g, p->beta, p->D, p->x};
    for (const void* v : words)
        if (!aligned(v, 4)) return SSM_ERR_INVALID_ARGUMENT;
    const int64_t strides[] = {p->q_stride, p->q_group, p->q_key,    p->k_stride, p->k_group,     p->k_key,
                               p->v_stride, p->v_head,  p->v_value,  p->y_stride, p->y_head,      p->y_value,
                               p->g_stride, p->g_head,  p->beta_stride, p->beta_head};
    for (int64_t s : strides)
        if (s < 0) return SSM_ERR_INVALID_ARGUMENT;
    if ((p->y_stride == 0 && p->Bsz > 1) || (p->y_head == 0 && p->H > 1) || (p->y_value == 0 && p->P > 1))
        return SSM_ERR_INVALID_ARGUMENT;
    for (int64_t s : strides)
        if (s >= ((int64_t)1 << 32)) return SSM_ERR_UNSUPPORTED;
    if (p->slots && p->n_slots > ((int64_t)1 << 40) / p->H) return SSM_ERR_UNSUPPORTED;
    LinearStepArgs a;
    a.Bsz = p->Bsz, a.H = p->H, a.G = p->G, a.N = p->N, a.P = p->P;
    a.scale = p->scale;
    a.slots = p->slots;
    a.n_slots = p->slots ? p->n_slots : p->Bsz;
    a.q = p->q, a.k = p->k, a.v = p->v, a.y = p->y;
    a.q_row = p->q_stride, a.q_group = p->q_group, a.q_key = p->q_key;
    a.k_row = p->k_stride, a.k_group = p->k_group, a.k_key = p->k_key;
    a.v_row = p->v_stride, a.v_head = p->v_head, a.v_value = p->v_value;
    a.y_row = p->y_stride, a.y_head = p->y_head, a.y_value = p->y_value;
    a.g = p->g, a.beta = p->beta;
    a.g_row = p->g_stride, a.g_head = p->g_head, a.beta_row = p->beta_stride, a.beta_head = p->beta_head;
    a.D = p->D, a.x = p->x;
    return device_status(launch_linear_step(p->dtype, a, (hipStream_t)stream));
}

}  // extern "C"

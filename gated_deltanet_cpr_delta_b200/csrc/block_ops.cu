// block_ops.cu -- host side of the norm of queries and keys with the position rotation, and of
// the clipped policy loss (gdn_cpr.h).
//
// As layer_ops.cu: it validates on the host, carves the caller's workspace and
// enqueues on the caller's stream; it allocates nothing, keeps no state and
// never synchronises.
#include "layer_host.cuh"
#include "k_policy.cuh"
#include "k_qknorm.cuh"

#include <cmath>

namespace {

// ------------------------------------------------------------- norm of queries and keys

gdn_status_t qk_check(const gdn_qk_norm_t* s)
{
    if (s == nullptr || s->tokens < 0 || s->tokens > kMaxRows || s->q_heads <= 0 || s->k_heads <= 0 || s->head_dim <= 0 ||
        s->rot_dim < 0 || s->rot_dim > s->head_dim || !(s->eps >= 0.0f) || !dtype_ok(s->in_dtype) || !dtype_ok(s->w_dtype))
        return GDN_ERR_INVALID_ARG;
    if (s->head_dim % 2 != 0 || s->rot_dim % 2 != 0 || s->head_dim > 256) return GDN_ERR_UNSUPPORTED;
    const size_t ws = esize(s->w_dtype);
    if ((s->q_weight && !aligned(s->q_weight, ws)) || (s->k_weight && !aligned(s->k_weight, ws))) return GDN_ERR_INVALID_ARG;
    if (s->rot_dim > 0 && (s->inv_freq == nullptr || !aligned(s->inv_freq, 4))) return GDN_ERR_INVALID_ARG;
    const int64_t heads = (int64_t)s->q_heads + s->k_heads;
    if (heads * s->head_dim > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (s->tokens == 0) return GDN_OK;
    if (s->rot_dim > 0 && (s->positions == nullptr || !aligned(s->positions, 4))) return GDN_ERR_INVALID_ARG;
    if (!rows_ok(s->q, s->q_stride, (int64_t)s->q_heads * s->head_dim, s->in_dtype) ||
        !rows_ok(s->k, s->k_stride, (int64_t)s->k_heads * s->head_dim, s->in_dtype))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Whether a thread's four pairs of a row are two accesses of four elements.
bool qk_vectors(const gdn_qk_norm_t* s, const void* p, int64_t stride, gdn_dtype_t t)
{
    const size_t bytes = 4 * esize(t);
    return aligned(p, bytes) && stride % 4 == 0 && s->head_dim % 8 == 0 && (s->interleaved || s->rot_dim % 8 == 0);
}

// Lanes of a row: a power of two that covers its pairs, four per lane.
int qk_lanes(int32_t d)
{
    int n = 1;
    while (n * 8 < d) n *= 2;
    return n;
}

// Tokens that a block takes at a time: the same number of tiles for every block, as large as 16 KB of angles (or
// 1024 rows) allow.  Each tile costs its setup and two barriers: 4 tokens at a time took 65 us where these took 63 (16384
// tokens, 16 + 16 heads of 128), the gradients 217 and 192 (32 + 32 heads).
int qk_tokens(const gdn_qk_norm_t* s, int tpr, int blocks)
{
    const int64_t heads = (int64_t)s->q_heads + s->k_heads;
    int64_t most = std::max<int64_t>(1, 1024 / heads);
    if (s->rot_dim > 0) most = std::min<int64_t>(most, 16 * 1024 / (32 * tpr));
    const int64_t rounds = std::max<int64_t>(1, ceil_div(s->tokens, most * blocks));
    return (int)std::max<int64_t>(1, ceil_div(s->tokens, rounds * blocks));
}

constexpr int kQkParts = 1024;  // most blocks of the backward (fewer than SMs where they share tiles)

// Blocks that share a tile's rows: where there are fewer tiles than SMs, as many as have two rows per thread.
unsigned qk_shares(const gdn::QkArgs& a, int64_t tiles, int sms)
{
    const int64_t rows = (int64_t)a.tokens * std::max(a.H[0], a.H[1]), slots = gdn::kQkThreads / a.tpr;
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(sms / std::max<int64_t>(1, tiles), rows / (2 * slots)));
}

template <typename T, typename G, bool BWD, bool VEC, bool INTER>
gdn_status_t qk_launch(gdn::QkArgs& a, dim3 blocks, cudaStream_t st)
{
    const size_t angles = a.rot > 0 ? sizeof(float) * 8 * (size_t)a.tokens * a.tpr : 0, weights = sizeof(float) * 16 * a.tpr;
    const size_t own = (angles + weights + 127) / 128 * 128;
    const size_t ring = VEC ? gdn::QkRing<T, G, gdn::qk_rows(BWD, sizeof(T)), BWD>::BYTES : 0;
    const size_t smem = std::max(own + ring, BWD ? sizeof(float) * (gdn::kQkThreads / 32) * a.d : 0);
    a.ring = (int32_t)own;
    auto k = gdn::k_qk_norm<T, G, VEC, INTER, BWD>;
    if (!raise_smem(k, smem)) return GDN_ERR_CUDA;
    return launch_next(k, blocks, dim3(gdn::kQkThreads), smem, 0, st, a) ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, typename G, bool BWD>
gdn_status_t qk_dispatch(gdn::QkArgs& a, bool vec, dim3 blocks, cudaStream_t st)
{
    if (vec) return a.interleaved ? qk_launch<T, G, BWD, true, true>(a, blocks, st) : qk_launch<T, G, BWD, true, false>(a, blocks, st);
    return a.interleaved ? qk_launch<T, G, BWD, false, true>(a, blocks, st) : qk_launch<T, G, BWD, false, false>(a, blocks, st);
}

gdn::QkArgs qk_args(const gdn_qk_norm_t* s, int blocks)
{
    gdn::QkArgs a{};
    a.x[0] = s->q; a.x[1] = s->k; a.ldx[0] = s->q_stride; a.ldx[1] = s->k_stride;
    a.w[0] = s->q_weight; a.w[1] = s->k_weight; a.H[0] = s->q_heads; a.H[1] = s->k_heads;
    a.w_bf16 = s->w_dtype == GDN_BF16; a.interleaved = s->interleaved != 0;
    a.pos = s->positions; a.freq = s->inv_freq; a.eps = s->eps;
    a.inv_n = s->unit ? 1.0f : 1.0f / (float)s->head_dim;
    a.T = s->tokens; a.d = s->head_dim; a.rot = s->rot_dim; a.tpr = qk_lanes(s->head_dim);
    a.tokens = qk_tokens(s, a.tpr, blocks);
    return a;
}

// ------------------------------------------------------------- policy loss

gdn_status_t policy_check(const gdn_policy_t* s, const int32_t* status)
{
    if (s == nullptr || s->rows < 0 || s->rows > kMaxRows || s->vocab <= 0 || !dtype_ok(s->in_dtype) || !aligned(status, 4))
        return GDN_ERR_INVALID_ARG;
    // (2^-100: the kernel's power of two for far logits stays in range)
    if (!(s->temperature >= 0x1p-100f) || std::isinf(s->temperature)) return GDN_ERR_INVALID_ARG;
    if ((s->old_logprob == nullptr) != (s->advantages == nullptr) || (s->ref_logprob && !s->old_logprob))
        return GDN_ERR_INVALID_ARG;
    if (s->old_logprob && (!(s->clip_low >= 0.0f) || !(s->clip_low <= 1.0f) || !(s->clip_high >= 0.0f) || std::isnan(s->kl_coef)))
        return GDN_ERR_INVALID_ARG;
    if (s->vocab > kMaxRows) return GDN_ERR_INVALID_ARG;
    if (!aligned(s->old_logprob, 4) || !aligned(s->ref_logprob, 4) || !aligned(s->advantages, 4)) return GDN_ERR_INVALID_ARG;
    if (s->rows == 0) return GDN_OK;
    if (!rows_ok(s->logits, s->logits_stride, s->vocab, s->in_dtype) || s->targets == nullptr || !aligned(s->targets, 8))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// A cluster of S blocks for each row, two blocks per SM.
template <typename T, bool BWD, bool ALIGNED>
gdn_status_t policy_split(const gdn::PolicyArgs& a, int S, cudaStream_t st)
{
    auto k = gdn::k_policy<T, BWD, ALIGNED, 256, 2, true>;
    constexpr size_t smem = (size_t)gdn::policy_slots(2) * gdn::policy_slot_bytes(256) + sizeof(float2) * 256 * (gdn::kPolicyParts / 2);
    if (!raise_smem<smem>(k)) return GDN_ERR_CUDA;
    return launch_next(k, dim3((unsigned)(a.T * S)), dim3(256 + 32), smem, S, st, a) ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, bool BWD, bool ALIGNED, int NT, int RES>
gdn_status_t policy_run(const gdn::PolicyArgs& a, cudaStream_t st)
{
    const int sms = sm_count();
    if (sms == 0) return GDN_ERR_CUDA;
    if constexpr (NT == 256) {
        const int64_t tile = gdn::policy_tile_bytes(NT) / (int64_t)sizeof(T);
        int S = 1 << gdn::policy_parts_log((int)ceil_div(a.V, tile));
        // One wave, and clusters of more than 2 leave some SMs out: 74 x 131072 bf16 takes 14.4 us with 4 blocks for each row
        // (all slots) and 10.7 with 2; with gradient 148 rows take 19 us with 2 and 23 with one.
        while (S > 1 && a.T * S > (S > 2 ? sms * 7 / 4 : sms * 2)) S /= 2;
        if (S > 1) return policy_split<T, BWD, ALIGNED>(a, S, st);
    }
    auto k = gdn::k_policy<T, BWD, ALIGNED, NT, RES, false>;
    constexpr size_t smem = (size_t)gdn::policy_slots(RES) * gdn::policy_slot_bytes(NT);
    if (!raise_smem<smem>(k)) return GDN_ERR_CUDA;
    const dim3 grid((unsigned)std::min<int64_t>(a.T, (int64_t)sms * RES));
    return launch_next(k, grid, dim3(NT + 32), smem, 0, st, a) ? GDN_OK : GDN_ERR_CUDA;
}

// Rows of up to two tiles of 4 KB by 64 threads, longer ones by 256 (the log-probabilities' bits
// follow from the vocabulary and the type).  Three blocks per SM, but two with larger rings where the rows that are walked at
// a time, of which a part is fetched again for the gradient, would not stay in L2: 4096 x 131072 bf16 (256 KB
// a row) 401 us with two, 459 with three; 4096 x 50021 199 and 180; 16384 x 32768 401 and 367.
template <typename T, bool BWD>
gdn_status_t policy_launch(const gdn::PolicyArgs& a, gdn_dtype_t t, cudaStream_t st)
{
    const bool whole = wide(a.z, a.ldz, a.V, t) && wide(a.dz, a.V, a.V, t);
    const int64_t bytes = (int64_t)a.V * (int64_t)sizeof(T);
    if (bytes <= 2 * gdn::policy_tile_bytes(64))
        return whole ? policy_run<T, BWD, true, 64, 8>(a, st) : policy_run<T, BWD, false, 64, 8>(a, st);
    if constexpr (BWD) {
        if (bytes > 160 * 1024)
            return whole ? policy_run<T, BWD, true, 256, 2>(a, st) : policy_run<T, BWD, false, 256, 2>(a, st);
    }
    return whole ? policy_run<T, BWD, true, 256, 3>(a, st) : policy_run<T, BWD, false, 256, 3>(a, st);
}

gdn::PolicyArgs policy_args(const gdn_policy_t* s, int32_t* status)
{
    gdn::PolicyArgs a{};
    a.z = s->logits; a.ldz = s->logits_stride; a.y = s->targets;
    a.old = s->old_logprob; a.ref = s->ref_logprob; a.adv = s->advantages;
    a.lo = 1.0f - s->clip_low; a.hi = 1.0f + s->clip_high; a.kl = s->kl_coef;
    a.c = (float)(1.4426950408889634 / (double)s->temperature); a.inv_tau = (float)(1.0 / (double)s->temperature);
    a.T = s->rows; a.V = s->vocab; a.status = status;
    return a;
}

}  // namespace

extern "C" {

gdn_status_t gdn_qk_norm_forward(const gdn_qk_norm_t* args, void* q_out, void* k_out, void* stream)
{
    const gdn_status_t bad = qk_check(args);
    if (bad != GDN_OK) return bad;
    const gdn_qk_norm_t& s = *args;
    if (s.tokens == 0) return GDN_OK;
    const int64_t T = s.tokens, wq = (int64_t)s.q_heads * s.head_dim, wk = (int64_t)s.k_heads * s.head_dim;
    if (!rows_ok(q_out, wq, wq, s.in_dtype) || !rows_ok(k_out, wk, wk, s.in_dtype)) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype), ws = esize(s.w_dtype);
    if (overlap({{q_out, T * wq, es}, {k_out, T * wk, es}},
                {{s.q, T, s.q_stride, wq, es}, {s.k, T, s.k_stride, wk, es}, {s.q_weight, s.head_dim, ws},
                 {s.k_weight, s.head_dim, ws}, {s.rot_dim ? s.positions : nullptr, T, 4},
                 {s.rot_dim ? s.inv_freq : nullptr, s.rot_dim / 2, 4}}))
        return GDN_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return GDN_ERR_CUDA;
    const gdn_dtype_t t = s.in_dtype;
    const bool vec = qk_vectors(args, s.q, s.q_stride, t) && qk_vectors(args, s.k, s.k_stride, t) &&
                     qk_vectors(args, q_out, wq, t) && qk_vectors(args, k_out, wk, t);
    const int most = sms * gdn::qk_resident(false, vec);
    gdn::QkArgs a = qk_args(args, most);
    a.out[0] = q_out; a.out[1] = k_out;
    const int64_t tiles = ceil_div(T, a.tokens);
    const dim3 blocks((unsigned)std::min<int64_t>(tiles, most), qk_shares(a, tiles, sms));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return t == GDN_BF16 ? qk_dispatch<__nv_bfloat16, __nv_bfloat16, false>(a, vec, blocks, st)
                         : qk_dispatch<float, float, false>(a, vec, blocks, st);
}

size_t gdn_qk_norm_backward_workspace_size(int64_t tokens, int32_t head_dim)
{
    if (tokens < 0 || head_dim <= 0) return 0;
    return align_up(sizeof(float) * 2 * (size_t)kQkParts * head_dim);
}

gdn_status_t gdn_qk_norm_backward(const gdn_qk_norm_t* args, const void* dq_out, int64_t dq_out_stride, const void* dk_out,
                                  int64_t dk_out_stride, void* dq, void* dk, float* dq_weight, float* dk_weight,
                                  void* workspace, size_t workspace_bytes, void* stream)
{
    return gdn_qk_norm_backward_ex(args, args != nullptr ? args->in_dtype : GDN_F32, dq_out, dq_out_stride, dk_out, dk_out_stride, dq, dk,
                                   dq_weight, dk_weight, workspace, workspace_bytes, stream);
}

gdn_status_t gdn_qk_norm_backward_ex(const gdn_qk_norm_t* args, gdn_dtype_t grad_dtype, const void* dq_out, int64_t dq_out_stride,
                                     const void* dk_out, int64_t dk_out_stride, void* dq, void* dk, float* dq_weight,
                                     float* dk_weight, void* workspace, size_t workspace_bytes, void* stream)
{
    const gdn_status_t bad = qk_check(args);
    if (bad != GDN_OK) return bad;
    if (!dtype_ok(grad_dtype)) return GDN_ERR_INVALID_ARG;
    if (grad_dtype != args->in_dtype && grad_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
    const gdn_qk_norm_t& s = *args;
    const int64_t T = s.tokens, wq = (int64_t)s.q_heads * s.head_dim, wk = (int64_t)s.k_heads * s.head_dim;
    const bool weights = dq_weight != nullptr || dk_weight != nullptr;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || (dq_weight && !s.q_weight) || (dk_weight && !s.k_weight))
        return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!rows_ok(dq_out, dq_out_stride, wq, grad_dtype) || !rows_ok(dk_out, dk_out_stride, wk, grad_dtype) ||
                  !rows_ok(dq, wq, wq, s.in_dtype) || !rows_ok(dk, wk, wk, s.in_dtype)))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype), ges = esize(grad_dtype), ws = esize(s.w_dtype);
    const size_t need = weights ? gdn_qk_norm_backward_workspace_size(T, s.head_dim) : 0;
    if (overlap({{dq, T * wq, es}, {dk, T * wk, es}, {dq_weight, s.head_dim, 4}, {dk_weight, s.head_dim, 4},
                 {workspace, (int64_t)need, 1}},
                {{s.q, T, s.q_stride, wq, es}, {s.k, T, s.k_stride, wk, es}, {dq_out, T, dq_out_stride, wq, ges},
                 {dk_out, T, dk_out_stride, wk, ges}, {s.q_weight, s.head_dim, ws}, {s.k_weight, s.head_dim, ws},
                 {s.rot_dim ? s.positions : nullptr, T, 4}, {s.rot_dim ? s.inv_freq : nullptr, s.rot_dim / 2, 4}}))
        return GDN_ERR_INVALID_ARG;
    if (weights && (workspace == nullptr || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (weights && !aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int64_t parts = 0;
    float* part = weights ? static_cast<float*>(workspace) : nullptr;
    if (T > 0) {
        const int sms = sm_count();
        if (sms == 0) return GDN_ERR_CUDA;
        gdn::QkArgs a = qk_args(args, (int)std::min<int64_t>(kQkParts, (int64_t)sms * gdn::qk_resident(true, true)));
        a.dy[0] = dq_out; a.dy[1] = dk_out; a.lddy[0] = dq_out_stride; a.lddy[1] = dk_out_stride;
        a.out[0] = dq; a.out[1] = dk; a.part = part;
        const int64_t tiles = ceil_div(T, a.tokens);
        const dim3 blocks((unsigned)std::min<int64_t>(tiles, std::min<int64_t>(kQkParts, (int64_t)sms * gdn::qk_resident(true, true))),
                          qk_shares(a, tiles, sms));
        parts = (int64_t)blocks.x * blocks.y;
        const gdn_dtype_t t = s.in_dtype;
        const bool vec = qk_vectors(args, s.q, s.q_stride, t) && qk_vectors(args, s.k, s.k_stride, t) &&
                         qk_vectors(args, dq_out, dq_out_stride, grad_dtype) && qk_vectors(args, dk_out, dk_out_stride, grad_dtype) &&
                         qk_vectors(args, dq, wq, t) && qk_vectors(args, dk, wk, t);
        const gdn_status_t r = t == GDN_F32 ? qk_dispatch<float, float, true>(a, vec, blocks, st)
                               : grad_dtype == GDN_F32 ? qk_dispatch<__nv_bfloat16, float, true>(a, vec, blocks, st)
                                                       : qk_dispatch<__nv_bfloat16, __nv_bfloat16, true>(a, vec, blocks, st);
        if (r != GDN_OK) return r;
    }
    if (!weights) return GDN_OK;
    const int64_t M = 2 * (int64_t)s.head_dim;
    return launch_next(gdn::k_colsum<gdn::QkGradMap>, dim3((unsigned)ceil_div(M, 32)), dim3(32, 8), 0, 0, st, part, parts, M,
                       gdn::QkGradMap{dq_weight, dk_weight, s.head_dim}) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_policy_loss_forward(const gdn_policy_t* args, float* loss, float* logprob, int32_t* status, void* stream)
{
    const gdn_status_t bad = policy_check(args, status);
    if (bad != GDN_OK) return bad;
    const gdn_policy_t& s = *args;
    if ((loss == nullptr) != (s.old_logprob == nullptr) || !aligned(loss, 4) || !aligned(logprob, 4)) return GDN_ERR_INVALID_ARG;
    if (s.rows == 0) return GDN_OK;
    if (logprob == nullptr) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype);
    if (overlap({{loss, s.rows, 4}, {logprob, s.rows, 4}, {status, 1, 4}},
                {{s.logits, s.rows, s.logits_stride, s.vocab, es}, {s.targets, s.rows, 8}, {s.old_logprob, s.rows, 4},
                 {s.ref_logprob, s.rows, 4}, {s.advantages, s.rows, 4}}))
        return GDN_ERR_INVALID_ARG;
    gdn::PolicyArgs a = policy_args(args, status);
    a.loss = loss; a.lp = logprob;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return s.in_dtype == GDN_BF16 ? policy_launch<__nv_bfloat16, false>(a, s.in_dtype, st)
                                  : policy_launch<float, false>(a, s.in_dtype, st);
}

gdn_status_t gdn_policy_loss_backward(const gdn_policy_t* args, const float* dloss, void* dlogits, float* loss,
                                      float* logprob, int32_t* status, void* stream)
{
    const gdn_status_t bad = policy_check(args, status);
    if (bad != GDN_OK) return bad;
    const gdn_policy_t& s = *args;
    if (s.old_logprob == nullptr || !aligned(loss, 4) || !aligned(logprob, 4) || !aligned(dloss, 4)) return GDN_ERR_INVALID_ARG;
    if (s.rows == 0) return GDN_OK;
    if (dloss == nullptr || !rows_ok(dlogits, s.vocab, s.vocab, s.in_dtype)) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype);
    // the gradient may take the place of dense logits: a row is on the chip before it is written
    const bool in_place = dlogits == s.logits && (s.logits_stride == s.vocab || s.rows == 1);
    if (overlap({{dlogits, s.rows * s.vocab, es}, {loss, s.rows, 4}, {logprob, s.rows, 4}, {status, 1, 4}},
                {{in_place ? nullptr : s.logits, s.rows, s.logits_stride, s.vocab, es}, {s.targets, s.rows, 8},
                 {s.old_logprob, s.rows, 4}, {s.ref_logprob, s.rows, 4}, {s.advantages, s.rows, 4}, {dloss, s.rows, 4}}))
        return GDN_ERR_INVALID_ARG;
    gdn::PolicyArgs a = policy_args(args, status);
    a.loss = loss; a.lp = logprob; a.dloss = dloss; a.dz = dlogits;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return s.in_dtype == GDN_BF16 ? policy_launch<__nv_bfloat16, true>(a, s.in_dtype, st)
                                  : policy_launch<float, true>(a, s.in_dtype, st);
}

}  // extern "C"

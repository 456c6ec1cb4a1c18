// layer_ops.cu -- host side of the layer operators of gdn_cpr.h: the short
// causal convolution, the selective state space scan and layer norm.
//
// As gdn_cpr.cu: it validates on the host, carves the caller's workspace and
// enqueues on the caller's stream; it allocates nothing, keeps no state and
// never synchronises.
#include "gdn_cpr.h"
#include "layer_host.cuh"
#include "k_conv.cuh"
#include "k_norm.cuh"
#include "k_ssm.cuh"
#include "k_ssm_bwd.cuh"

namespace {

using gdn::Seqs;

// ------------------------------------------------------------------- convolution

// Threads along the channels of a 128-thread block: a power of two that covers
// the channels' vectors, so that narrow tensors fill their blocks with token runs.
int conv_cx(int64_t nvec)
{
    int cx = 8;
    while (cx < 128 && cx < nvec) cx *= 2;
    return cx;
}

// Tokens per run.  A run reads W - 1 rows of its neighbour again, loads the taps and
// (backward) leaves W + 1 partial sums per channel, so it is as long as one full wave of
// blocks allows (`resident` per SM), within [8, 512].
int conv_run(int64_t T, int64_t nvec, int sms, int resident)
{
    const int64_t threads = (int64_t)sms * resident * 128;
    const int64_t run = ceil_div(T * nvec, threads);
    return (int)std::max<int64_t>(8, std::min<int64_t>(512, ceil_div(run, 8) * 8));
}

// Grid of the convolution kernels for V channels per thread.
gdn_status_t conv_grid(gdn::ConvArgs& a, int V, int resident, unsigned* blocks)
{
    const int sms = sm_count();
    if (sms == 0) return GDN_ERR_CUDA;
    const int64_t nvec = ceil_div(a.D, V);
    a.cx = conv_cx(nvec);
    a.ncb = (int32_t)ceil_div(nvec, a.cx);
    a.run = conv_run(a.s.T, (int64_t)a.ncb * a.cx, sms, resident);
    const int ny = 128 / a.cx;
    a.ntiles = ceil_div(a.s.T, (int64_t)a.run * ny);
    const int64_t n = (a.ntiles + ceil_div(a.s.N, ny)) * a.ncb;
    if (n > INT32_MAX) return GDN_ERR_INVALID_ARG;
    *blocks = (unsigned)n;
    return GDN_OK;
}

// Rows of partial weight gradients for any vector width and any number of SMs:
// a tile holds at least 8 tokens.
int64_t conv_tiles_max(int64_t T) { return ceil_div(T, 8); }

template <typename T, int V>
void launch_conv_fwd(const gdn::ConvArgs& a, int W, unsigned blocks, cudaStream_t st)
{
    constexpr size_t sm = gdn::ConvRing<T, V, gdn::kConvAhead>::BYTES;
    if (W == 2) gdn::k_conv_fwd<T, 2, V><<<blocks, 128, sm, st>>>(a);
    else if (W == 3) gdn::k_conv_fwd<T, 3, V><<<blocks, 128, sm, st>>>(a);
    else gdn::k_conv_fwd<T, 4, V><<<blocks, 128, sm, st>>>(a);
}

template <typename T, int V>
void launch_conv_bwd(const gdn::ConvArgs& a, int W, unsigned blocks, cudaStream_t st)
{
    const size_t sm = std::max(2 * gdn::ConvRing<T, V, gdn::kConvAhead>::BYTES, sizeof(float) * (W + 1) * V * 128);
    if (W == 2) gdn::k_conv_bwd<T, 2, V><<<blocks, 128, sm, st>>>(a);
    else if (W == 3) gdn::k_conv_bwd<T, 3, V><<<blocks, 128, sm, st>>>(a);
    else gdn::k_conv_bwd<T, 4, V><<<blocks, 128, sm, st>>>(a);
}

template <typename T, int V>
void launch_conv_step(const void* x, int64_t ldx, const void* w, const void* b, const void* s, void* so, int64_t N,
                      int32_t D, int W, int silu, int wb, void* y, cudaStream_t st)
{
    const unsigned blocks = (unsigned)ceil_div(N * (D / V), 128);
    const T *tx = static_cast<const T*>(x), *ts = static_cast<const T*>(s);
    T *to = static_cast<T*>(so), *ty = static_cast<T*>(y);
    if (W == 2) gdn::k_conv_step<T, 2, V><<<blocks, 128, 0, st>>>(tx, ldx, w, b, ts, to, N, D, silu, wb, ty);
    else if (W == 3) gdn::k_conv_step<T, 3, V><<<blocks, 128, 0, st>>>(tx, ldx, w, b, ts, to, N, D, silu, wb, ty);
    else gdn::k_conv_step<T, 4, V><<<blocks, 128, 0, st>>>(tx, ldx, w, b, ts, to, N, D, silu, wb, ty);
}

gdn_status_t conv_check(const void* x, int64_t x_stride, const void* weight, const void* bias, const void* state,
                        const int32_t* cu, const int32_t* status, int32_t num_seqs, int64_t T, int32_t D, int32_t W,
                        gdn_dtype_t in, gdn_dtype_t wt)
{
    if (num_seqs < 0 || T < 0 || T > kMaxRows || D <= 0 || W <= 0) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(in) || !dtype_ok(wt)) return GDN_ERR_INVALID_ARG;
    if (W < 2 || W > 4) return GDN_ERR_UNSUPPORTED;
    if ((cu == nullptr && num_seqs != 1) || !aligned(cu, 4) || !aligned(status, 4)) return GDN_ERR_INVALID_ARG;
    if (T > 0 && !rows_ok(x, x_stride, D, in)) return GDN_ERR_INVALID_ARG;
    if (weight == nullptr || !aligned(weight, esize(wt)) || (bias && !aligned(bias, esize(wt))))
        return GDN_ERR_INVALID_ARG;
    if (state != nullptr && !aligned(state, 16)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// ------------------------------------------------------------------- layer norm

struct NormPlan {
    int V, NV, tpr, threads;
    bool wide;   // one block per row, the row read again
    bool shift;  // dense rows that are not whole vectors
};

// A row's threads: up to a warp with one vector each, then more vectors (up to
// `most`) before more threads, so that a row's sums cross few warps.
NormPlan norm_plan(int32_t D, int V, int most, int max_threads)
{
    NormPlan p{};
    const int64_t nvec = ceil_div(D, V);
    p.V = V;
    int tpr = 8;
    while (tpr < 32 && (int64_t)tpr < nvec) tpr *= 2;
    while (tpr < max_threads && (int64_t)tpr * most < nvec) tpr *= 2;
    p.tpr = tpr;
    const int64_t nv = ceil_div(nvec, tpr);
    p.NV = 1;
    while (p.NV < nv) p.NV *= 2;
    p.wide = p.NV > most;
    p.threads = std::max(tpr, 128);
    return p;
}

// Blocks that walk the rows: a full GPU of about `resident` threads per SM.
int64_t norm_blocks(int64_t rows, const NormPlan& p, int resident)
{
    const int64_t all = ceil_div(rows, p.threads / p.tpr);
    const int64_t most = (int64_t)148 * std::max(1, resident / p.threads);
    if (all <= most) return all;
    return p.shift ? most / p.V * p.V : most;  // shifted rows: a stride of whole vectors of rows
}

template <typename T, typename WT, int V, int NV>
bool norm_fwd_nv(const gdn::NormArgs& a, const NormPlan& p, cudaStream_t st)
{
    if (p.NV == NV) {
        const size_t sm = gdn::NormRing<T, V, NV, gdn::norm_depth(NV)>::BYTES * p.threads;
        const int resident = V == 1 ? 2048 : NV == 1 ? 1280 : NV == 2 ? 1024 : 512;
        auto k = gdn::k_norm_fwd<T, WT, V, NV, false>;
        if constexpr (V > 1)
            if (p.shift) k = gdn::k_norm_fwd<T, WT, V, NV, true>;
        if (!raise_smem(k, sm)) return false;
        k<<<(unsigned)norm_blocks(a.R, p, resident), p.threads, sm, st>>>(a);
    } else if constexpr (NV < (V == 1 ? 16 : 4)) {
        return norm_fwd_nv<T, WT, V, NV * 2>(a, p, st);
    }
    return launched();
}

template <typename T, int V>
bool launch_norm_fwd(const gdn::NormArgs& a, const NormPlan& p, cudaStream_t st)
{
    return a.w_bf16 ? norm_fwd_nv<T, __nv_bfloat16, V, 1>(a, p, st) : norm_fwd_nv<T, float, V, 1>(a, p, st);
}

template <typename T, typename WT, int V, int NV>
bool norm_bwd_nv(const gdn::NormArgs& a, const NormPlan& p, int64_t* blocks, cudaStream_t st)
{
    if (p.NV == NV) {
        const size_t sm = std::max(2 * gdn::NormRing<T, V, NV, gdn::norm_depth(NV)>::BYTES * p.threads,
                                   p.threads > p.tpr ? sizeof(float) * 2 * (size_t)a.D : 0);
        auto k = gdn::k_norm_bwd<T, WT, V, NV, false>;
        if constexpr (V > 1)
            if (p.shift) k = gdn::k_norm_bwd<T, WT, V, NV, true>;
        if (!raise_smem(k, sm)) return false;
        *blocks = norm_blocks(a.R, p, NV == 1 && V > 1 ? 1024 : 512);
        k<<<(unsigned)*blocks, p.threads, sm, st>>>(a);
    } else if constexpr (NV < (V == 1 ? 16 : 4)) {
        return norm_bwd_nv<T, WT, V, NV * 2>(a, p, blocks, st);
    }
    return launched();
}

// *blocks: how many shares of dw and db it leaves
template <typename T, int V>
bool launch_norm_bwd(const gdn::NormArgs& a, const NormPlan& p, int64_t* blocks, cudaStream_t st)
{
    return a.w_bf16 ? norm_bwd_nv<T, __nv_bfloat16, V, 1>(a, p, blocks, st) : norm_bwd_nv<T, float, V, 1>(a, p, blocks, st);
}

constexpr int64_t kNormParts = 148 * 8;  // most blocks that keep a share of dw and db (1024 threads per SM, 128 to a block)
int64_t norm_parts(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, kNormParts)); }

// ------------------------------------------------------------------- scan

// Tokens per chunk of the backward: about 32 warps per SM over the whole batch, at least 64.
// T or more means that no sequence is cut.
int64_t ssm_bwd_chunk(int64_t T, int32_t D, int32_t S)
{
    const int64_t across = ceil_div(D, 2 * 128 / S);  // warps that walk one sequence
    const int64_t chunks = std::max<int64_t>(1, 148 * 32 / across);
    return std::max<int64_t>(64, ceil_div(ceil_div(T, chunks), gdn::kSsmSave) * gdn::kSsmSave);
}

struct SsmWorkspace {
    float *ebuf, *dsum, *partA, *partD, *partBC;
    size_t bytes;
};

SsmWorkspace ssm_carve(void* base, int64_t T, int32_t N, int32_t D, int32_t G, int32_t S)
{
    SsmWorkspace w{};
    size_t off = 0;
    char* b = static_cast<char*>(base);
    auto take = [&](size_t floats) {
        float* p = b != nullptr ? reinterpret_cast<float*>(b + off) : nullptr;
        off = align_up(off + sizeof(float) * floats);
        return p;
    };
    const int64_t Lc = ssm_bwd_chunk(T, D, S), cpg = ceil_div(D / G, 2 * 128 / S * 4);
    const size_t slots = (size_t)(T / Lc + N), per = (size_t)D * S;
    if (T > Lc) {
        w.ebuf = take(slots * per);
        w.dsum = take(slots * D);
    }
    w.partA = take(slots * per);
    w.partD = take(slots * 2 * D);
    w.partBC = take((size_t)cpg * T * G * 2 * S);
    w.bytes = std::max<size_t>(off, kAlign);
    return w;
}

gdn_status_t ssm_check(const gdn_ssm_t* s, const int32_t* status, bool step)
{
    if (s == nullptr || !aligned(status, 4)) return GDN_ERR_INVALID_ARG;
    if (s->num_seqs < 0 || s->total_tokens < 0 || s->total_tokens > kMaxRows || s->channels <= 0 ||
        s->channels > kMaxRows || s->groups <= 0 || s->states <= 0 || s->channels % s->groups != 0)
        return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(s->in_dtype)) return GDN_ERR_INVALID_ARG;
    if (s->states != 16 && s->states != 32 && s->states != 64) return GDN_ERR_UNSUPPORTED;
    if (s->A == nullptr || !aligned(s->A, 16)) return GDN_ERR_INVALID_ARG;
    if ((s->D && !aligned(s->D, 4)) || (s->dt_bias && !aligned(s->dt_bias, 4))) return GDN_ERR_INVALID_ARG;
    if (step ? s->total_tokens != s->num_seqs
             : (s->cu_seqlens == nullptr && s->num_seqs != 1) || !aligned(s->cu_seqlens, 4))
        return GDN_ERR_INVALID_ARG;
    if (s->total_tokens > 0) {
        const int64_t bc = (int64_t)s->groups * s->states;
        if (!rows_ok(s->x, s->x_stride, s->channels, s->in_dtype) ||
            !rows_ok(s->dt, s->dt_stride, s->channels, s->in_dtype) || !rows_ok(s->B, s->B_stride, bc, s->in_dtype) ||
            !rows_ok(s->C, s->C_stride, bc, s->in_dtype) ||
            (s->z != nullptr && !rows_ok(s->z, s->z_stride, s->channels, s->in_dtype)))
            return GDN_ERR_INVALID_ARG;
    }
    return GDN_OK;
}

gdn::SsmArgs ssm_args(const gdn_ssm_t* s, int block_channels)
{
    gdn::SsmArgs a{};
    a.s = Seqs{s->cu_seqlens, s->num_seqs, s->total_tokens};
    a.x = s->x; a.dt = s->dt; a.z = s->z; a.B = s->B; a.C = s->C;
    a.ldx = s->x_stride; a.lddt = s->dt_stride; a.ldz = s->z_stride; a.ldB = s->B_stride; a.ldC = s->C_stride;
    a.A = s->A; a.Dp = s->D; a.dt_bias = s->dt_bias;
    a.D = s->channels; a.G = s->groups; a.Dg = s->channels / s->groups;
    a.cpg = (int32_t)ceil_div(a.Dg, block_channels);
    a.softplus = s->delta_softplus != 0;
    a.bc16 = wide(s->B, s->B_stride, s->states, s->in_dtype) && wide(s->C, s->C_stride, s->states, s->in_dtype);
    return a;
}

// All token tensors in 16-byte accesses (a group's channels have to be whole vectors).
bool ssm_wide(const gdn_ssm_t* s)
{
    const int64_t Dg = s->channels / s->groups;
    const int64_t v = 16 / (int64_t)esize(s->in_dtype);
    return Dg % v == 0 && wide(s->x, s->x_stride, Dg, s->in_dtype) && wide(s->dt, s->dt_stride, Dg, s->in_dtype) &&
           wide(s->z, s->z_stride, Dg, s->in_dtype);
}

template <typename T, int S, int V, int SEG>
gdn_status_t ssm_forward_seg(gdn::SsmArgs a, cudaStream_t st)
{
    using Cf = gdn::SsmFwdCfg<T, S, SEG>;
    a.cpg = (int32_t)ceil_div(a.Dg, Cf::CB);
    const int64_t blocks = (int64_t)a.s.N * a.G * a.cpg;
    if (blocks > INT32_MAX) return GDN_ERR_INVALID_ARG;
    auto k = gdn::k_ssm_fwd<T, S, V, SEG>;
    if (!raise_smem<Cf::BYTES>(k)) return GDN_ERR_CUDA;
    k<<<(unsigned)blocks, Cf::THREADS, Cf::BYTES, st>>>(a);
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, int S, int V>
gdn_status_t ssm_forward_launch(const gdn::SsmArgs& a, cudaStream_t st)
{
    // Tiles of 64 tokens (8 segments, 4 channels per warp) or of 128 (16 segments, 2 channels per
    // warp: twice the blocks, half the steps of a sequence, more shared memory).  16 where its
    // blocks take at most three rounds of those that are resident.  Measured, 8 against 16 segments, bf16:
    //   1 sequence x 2048 tokens x 1024 channels (0.2, 0.3 and 0.9 rounds at 16, 32 and 64 states):
    //     96 against 57, 160 against 94, 293 against 176 us
    //   4 x 2048 x 2048 (1.7, 2.3, 6.9): 176 against 181, 307 against 358, 733 against 1180 us
    //   8 x 2048 x 2048 (3.5, 4.6, 13.8): 303 against 344, 528 against 657, 1356 against 2348 us
    // The lengths are not known here.  In ragged batches the longest sequence counts, which 16 segments walk faster: 9
    // sequences of 1 to 1500 tokens x 777 channels (1.5, 2.0, 6.0): 152 against 99, 287 against 160, 434 against 447 us.
    const int sms = sm_count();
    if (sms == 0) return GDN_ERR_CUDA;
    using Cf = gdn::SsmFwdCfg<T, S, 16>;
    constexpr int64_t per_sm = std::min<int64_t>(4, 228 * 1024 / (Cf::BYTES + 1024));  // 4: launch bounds
    if ((int64_t)a.s.N * a.G * ceil_div(a.Dg, Cf::CB) > 3 * per_sm * sms) return ssm_forward_seg<T, S, V, 8>(a, st);
    return ssm_forward_seg<T, S, V, 16>(a, st);
}

template <typename T, int S, int V>
gdn_status_t ssm_backward_launch(const gdn::SsmBwdArgs& b, void* dB, void* dC, float* dA, float* dD, float* ddt_bias,
                                 cudaStream_t st)
{
    const gdn::SsmArgs& a = b.f;
    const int64_t slots = a.s.T / b.Lc + a.s.N;
    if (slots * a.G * a.cpg > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (a.s.T > b.Lc) {
        const int64_t rev = slots * a.G * ceil_div(a.Dg, gdn::SsmRevCfg<S>::CB);
        gdn::k_ssm_rev<T, S, V><<<(unsigned)rev, gdn::kSsmThreads, 0, st>>>(b);
        const int64_t ids = (int64_t)a.s.N * a.D * (S / 4);
        gdn::k_ssm_bwd_pass<S><<<(unsigned)ceil_div(ids, 128), 128, 0, st>>>(b);
    }
    constexpr size_t sm = gdn::SsmBwdCfg<S>::SMEM;
    auto k = a.z != nullptr ? gdn::k_ssm_bwd<T, S, V, true> : gdn::k_ssm_bwd<T, S, V, false>;
    if (!raise_smem<sm>(k)) return GDN_ERR_CUDA;
    k<<<(unsigned)(slots * a.G * a.cpg), gdn::kSsmThreads, sm, st>>>(b);
    if (a.s.T > 0) {
        const int64_t ids = a.s.T * a.G * 2 * S;
        gdn::k_ssm_dbc<T, S><<<(unsigned)ceil_div(ids, 256), 256, 0, st>>>(a.s, b.partBC, a.G, a.cpg,
                                                                           static_cast<T*>(dB), static_cast<T*>(dC));
    }
    const dim3 blk(32, 8);
    const int64_t mA = (int64_t)a.D * S, mD = 2 * (int64_t)a.D;
    gdn::k_colsum<<<(unsigned)ceil_div(mA, 32), blk, 0, st>>>(b.partA, slots, mA, gdn::PlainMap{dA});
    if (dD != nullptr || ddt_bias != nullptr)
        gdn::k_colsum<<<(unsigned)ceil_div(mD, 32), blk, 0, st>>>(b.partD, slots, mD,
                                                                  gdn::SsmGradMap{dD, ddt_bias, a.D});
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

// in_dtype, states and vector width as template arguments of f<T, S, V>(...)
#define SSM_DISPATCH(f, in_dtype, states, is_wide, ...)                                                        \
    do {                                                                                                       \
        if ((in_dtype) == GDN_BF16) {                                                                          \
            if ((states) == 16) return (is_wide) ? f<__nv_bfloat16, 16, 8>(__VA_ARGS__) : f<__nv_bfloat16, 16, 1>(__VA_ARGS__); \
            if ((states) == 32) return (is_wide) ? f<__nv_bfloat16, 32, 8>(__VA_ARGS__) : f<__nv_bfloat16, 32, 1>(__VA_ARGS__); \
            return (is_wide) ? f<__nv_bfloat16, 64, 8>(__VA_ARGS__) : f<__nv_bfloat16, 64, 1>(__VA_ARGS__);    \
        }                                                                                                      \
        if ((states) == 16) return (is_wide) ? f<float, 16, 4>(__VA_ARGS__) : f<float, 16, 1>(__VA_ARGS__);    \
        if ((states) == 32) return (is_wide) ? f<float, 32, 4>(__VA_ARGS__) : f<float, 32, 1>(__VA_ARGS__);    \
        return (is_wide) ? f<float, 64, 4>(__VA_ARGS__) : f<float, 64, 1>(__VA_ARGS__);                        \
    } while (0)

template <typename T, int S>
gdn_status_t ssm_step_launch(const gdn::SsmArgs& a, cudaStream_t st)
{
    const unsigned across = (unsigned)ceil_div(a.D, 1024 / S);
    for (int64_t n = 0; n < a.s.N; n += 65535) {  // a grid has at most 65535 rows
        gdn::SsmArgs b = a;
        const int64_t es = sizeof(T), per = (int64_t)a.D * S;
        b.x = static_cast<const char*>(a.x) + n * a.ldx * es;
        b.dt = static_cast<const char*>(a.dt) + n * a.lddt * es;
        b.z = a.z != nullptr ? static_cast<const char*>(a.z) + n * a.ldz * es : nullptr;
        b.B = static_cast<const char*>(a.B) + n * a.ldB * es;
        b.C = static_cast<const char*>(a.C) + n * a.ldC * es;
        b.state_in = a.state_in + n * per;
        b.state_out = a.state_out + n * per;
        b.y = static_cast<char*>(a.y) + n * (int64_t)a.D * es;
        gdn::k_ssm_step<T, S><<<dim3(across, (unsigned)std::min<int64_t>(65535, a.s.N - n)), 256, 0, st>>>(b);
    }
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

extern "C" {

gdn_status_t gdn_conv_forward(const void* x, int64_t x_stride, const void* weight, const void* bias,
                              const void* state_in, const int32_t* cu_seqlens, int32_t num_seqs,
                              int64_t total_tokens, int32_t channels, int32_t width, int32_t silu,
                              gdn_dtype_t in_dtype, gdn_dtype_t w_dtype, void* y, void* state_out, int32_t* status,
                              void* stream)
{
    const gdn_status_t bad = conv_check(x, x_stride, weight, bias, state_in, cu_seqlens, status, num_seqs, total_tokens,
                                        channels, width, in_dtype, w_dtype);
    if (bad != GDN_OK) return bad;
    if (num_seqs == 0) return GDN_OK;
    if (state_out == nullptr || !aligned(state_out, 16)) return GDN_ERR_INVALID_ARG;
    if (total_tokens > 0 && !rows_ok(y, channels, channels, in_dtype)) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(in_dtype);
    const int64_t tail = (int64_t)num_seqs * (width - 1) * channels;
    if (overlap({{y, total_tokens * channels, es}, {state_out, tail, es}, {status, 1, 4}},
                {{x, total_tokens, x_stride, channels, es}, {state_in, tail, es}, {cu_seqlens, num_seqs + 1LL, 4},
                 {weight, (int64_t)channels * width, esize(w_dtype)}, {bias, channels, esize(w_dtype)}}))
        return GDN_ERR_INVALID_ARG;
    gdn::ConvArgs a{};
    a.s = Seqs{cu_seqlens, num_seqs, total_tokens};
    a.x = x; a.ldx = x_stride; a.w = weight; a.bias = bias; a.state_in = state_in;
    a.D = channels; a.silu = silu != 0; a.w_bf16 = w_dtype == GDN_BF16;
    a.y = y; a.state_out = state_out; a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto can = [&](int64_t v) {
        return groups(x, x_stride, channels, in_dtype, v) && groups(y, channels, channels, in_dtype, v);
    };
    const int V = can(4) ? 4 : can(2) ? 2 : 1;  // channels per thread
    unsigned blocks = 0;
    const gdn_status_t grid = conv_grid(a, V, V == 4 ? 7 : 8, &blocks);
    if (grid != GDN_OK) return grid;
    if (in_dtype == GDN_BF16) {
        if (V == 4) launch_conv_fwd<__nv_bfloat16, 4>(a, width, blocks, st);
        else if (V == 2) launch_conv_fwd<__nv_bfloat16, 2>(a, width, blocks, st);
        else launch_conv_fwd<__nv_bfloat16, 1>(a, width, blocks, st);
    } else {
        if (V == 4) launch_conv_fwd<float, 4>(a, width, blocks, st);
        else if (V == 2) launch_conv_fwd<float, 2>(a, width, blocks, st);
        else launch_conv_fwd<float, 1>(a, width, blocks, st);
    }
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_conv_backward_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t channels, int32_t width)
{
    if (total_tokens < 0 || num_seqs < 0 || channels <= 0 || width < 2 || width > 4) return 0;
    return align_up(sizeof(float) * (size_t)std::max<int64_t>(1, conv_tiles_max(total_tokens)) * (width + 1) *
                    channels);
}

gdn_status_t gdn_conv_backward(const void* x, int64_t x_stride, const void* weight, const void* bias,
                               const void* state_in, const void* dy, int64_t dy_stride, const float* dstate_out,
                               const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t channels,
                               int32_t width, int32_t silu, gdn_dtype_t in_dtype, gdn_dtype_t w_dtype, void* dx,
                               float* dweight, float* dbias, float* dstate_in, void* workspace,
                               size_t workspace_bytes, int32_t* status, void* stream)
{
    const gdn_status_t bad = conv_check(x, x_stride, weight, bias, state_in, cu_seqlens, status, num_seqs, total_tokens,
                                        channels, width, in_dtype, w_dtype);
    if (bad != GDN_OK) return bad;
    if (dweight == nullptr || !aligned(dweight, 16) || (dbias && !aligned(dbias, 16))) return GDN_ERR_INVALID_ARG;
    if (num_seqs > 0 && (dstate_in == nullptr || !aligned(dstate_in, 16))) return GDN_ERR_INVALID_ARG;
    if (dstate_out != nullptr && !aligned(dstate_out, 16)) return GDN_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!rows_ok(dy, dy_stride, channels, in_dtype) || !rows_ok(dx, channels, channels, in_dtype)))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(in_dtype);
    const int64_t tail = (int64_t)num_seqs * (width - 1) * channels;
    const size_t need = gdn_conv_backward_workspace_size(total_tokens, num_seqs, channels, width);
    if (overlap({{dx, total_tokens * channels, es}, {dweight, (int64_t)channels * width, 4}, {dbias, channels, 4},
                 {dstate_in, tail, 4}, {workspace, (int64_t)need, 1}, {status, 1, 4}},
                {{x, total_tokens, x_stride, channels, es}, {dy, total_tokens, dy_stride, channels, es},
                 {state_in, tail, es}, {dstate_out, tail, 4}, {cu_seqlens, num_seqs + 1LL, 4},
                 {weight, (int64_t)channels * width, esize(w_dtype)}, {bias, channels, esize(w_dtype)}}))
        return GDN_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    gdn::ConvArgs a{};
    a.s = Seqs{cu_seqlens, num_seqs, num_seqs > 0 ? total_tokens : 0};
    a.x = x; a.ldx = x_stride; a.w = weight; a.bias = bias; a.state_in = state_in;
    a.D = channels; a.silu = silu != 0; a.w_bf16 = w_dtype == GDN_BF16;
    a.dy = dy; a.lddy = dy_stride; a.dstate_out = dstate_out; a.dx = dx; a.dstate_in = dstate_in;
    a.part = static_cast<float*>(workspace);
    a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto can = [&](int64_t v) {
        return groups(x, x_stride, channels, in_dtype, v) && groups(dy, dy_stride, channels, in_dtype, v) &&
               groups(dx, channels, channels, in_dtype, v);
    };
    const int V = can(4) ? 4 : can(2) ? 2 : 1;  // channels per thread
    unsigned blocks = 0;
    const gdn_status_t grid = conv_grid(a, V, 4, &blocks);
    if (grid != GDN_OK) return grid;
    if (blocks > 0) {
        if (in_dtype == GDN_BF16) {
            if (V == 4) launch_conv_bwd<__nv_bfloat16, 4>(a, width, blocks, st);
            else if (V == 2) launch_conv_bwd<__nv_bfloat16, 2>(a, width, blocks, st);
            else launch_conv_bwd<__nv_bfloat16, 1>(a, width, blocks, st);
        } else {
            if (V == 4) launch_conv_bwd<float, 4>(a, width, blocks, st);
            else if (V == 2) launch_conv_bwd<float, 2>(a, width, blocks, st);
            else launch_conv_bwd<float, 1>(a, width, blocks, st);
        }
    }
    const int64_t M = (int64_t)channels * (width + 1);
    gdn::k_colsum<<<(unsigned)ceil_div(M, 32), dim3(32, 8), 0, st>>>(a.part, a.ntiles, M,
                                                                     gdn::ConvGradMap{dweight, dbias, channels, width});
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_conv_step(const void* x, int64_t x_stride, const void* weight, const void* bias, const void* state,
                           void* state_out, int32_t num_seqs, int32_t channels, int32_t width, int32_t silu,
                           gdn_dtype_t in_dtype, gdn_dtype_t w_dtype, void* y, void* stream)
{
    static const int32_t none = 0;  // conv_check wants offsets for num_seqs != 1; the step reads none
    const gdn_status_t bad =
        conv_check(x, x_stride, weight, bias, state, &none, nullptr, num_seqs, num_seqs, channels, width, in_dtype, w_dtype);
    if (bad != GDN_OK) return bad;
    if (num_seqs == 0) return GDN_OK;
    if (state == nullptr || state_out == nullptr || !aligned(state_out, 16) || !rows_ok(y, channels, channels, in_dtype))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(in_dtype);
    const int64_t tail = (int64_t)num_seqs * (width - 1) * channels;
    if (overlap({{y, (int64_t)num_seqs * channels, es}, {state_out, tail, es}},
                {{x, num_seqs, x_stride, channels, es}, {state != state_out ? state : nullptr, tail, es},
                 {weight, (int64_t)channels * width, esize(w_dtype)}, {bias, channels, esize(w_dtype)}}))
        return GDN_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool v16 = wide(x, x_stride, channels, in_dtype) && wide(y, channels, channels, in_dtype);
    if (ceil_div((int64_t)num_seqs * (channels / (v16 ? 16 / (int)es : 1)), 128) > INT32_MAX) return GDN_ERR_INVALID_ARG;
    const int wb = w_dtype == GDN_BF16, sl = silu != 0;
    if (in_dtype == GDN_BF16) {
        if (v16) launch_conv_step<__nv_bfloat16, 8>(x, x_stride, weight, bias, state, state_out, num_seqs, channels, width, sl, wb, y, st);
        else launch_conv_step<__nv_bfloat16, 1>(x, x_stride, weight, bias, state, state_out, num_seqs, channels, width, sl, wb, y, st);
    } else {
        if (v16) launch_conv_step<float, 4>(x, x_stride, weight, bias, state, state_out, num_seqs, channels, width, sl, wb, y, st);
        else launch_conv_step<float, 1>(x, x_stride, weight, bias, state, state_out, num_seqs, channels, width, sl, wb, y, st);
    }
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_layer_norm_forward(const void* x, int64_t x_stride, const void* weight, const void* bias, float eps,
                                    int64_t rows, int32_t width, gdn_dtype_t in_dtype, gdn_dtype_t w_dtype, void* y,
                                    float* mean, float* rstd, void* stream)
{
    if (rows < 0 || rows > kMaxRows || width <= 0 || width > kMaxRows || !(eps >= 0.0f) || !dtype_ok(in_dtype) || !dtype_ok(w_dtype))
        return GDN_ERR_INVALID_ARG;
    if (weight == nullptr || !aligned(weight, esize(w_dtype)) || (bias && !aligned(bias, esize(w_dtype))))
        return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    if (!rows_ok(x, x_stride, width, in_dtype) || !rows_ok(y, width, width, in_dtype) || mean == nullptr ||
        rstd == nullptr || !aligned(mean, 4) || !aligned(rstd, 4))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(in_dtype);
    if (overlap({{y, rows * width, es}, {mean, rows, 4}, {rstd, rows, 4}},
                {{x, rows, x_stride, width, es}, {weight, width, esize(w_dtype)}, {bias, width, esize(w_dtype)}}))
        return GDN_ERR_INVALID_ARG;
    gdn::NormArgs a{};
    a.x = x; a.ldx = x_stride; a.w = weight; a.b = bias; a.w_bf16 = w_dtype == GDN_BF16;
    a.eps = eps; a.R = rows; a.D = width; a.y = y; a.mean = mean; a.rstd = rstd;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    bool v16 = wide(x, x_stride, width, in_dtype) && wide(y, width, width, in_dtype);
    const int vec = (int)(16 / es);
    const bool shift = !v16 && x_stride == width && aligned(x, 16) && aligned(y, 16) && width >= 4 * vec;
    v16 = v16 || shift;
    const int32_t span = shift ? width + vec - 1 : width;  // what the vectors of a row may cover
    // two vectors per thread measured best at 4096 x 16384 rows (63 us; four: 79, one: 101)
    NormPlan p = v16 ? norm_plan(span, vec, 2, 512) : norm_plan(width, 1, 16, 1024);
    if (p.wide && v16) p = norm_plan(span, vec, 4, 512);
    p.shift = shift;
    a.tpr = p.tpr;
    if (p.wide) {
        if (in_dtype == GDN_BF16) gdn::k_norm_fwd_wide<__nv_bfloat16><<<(unsigned)rows, 1024, 0, st>>>(a);
        else gdn::k_norm_fwd_wide<float><<<(unsigned)rows, 1024, 0, st>>>(a);
        return launched() ? GDN_OK : GDN_ERR_CUDA;
    }
    bool ok;
    if (in_dtype == GDN_BF16) ok = v16 ? launch_norm_fwd<__nv_bfloat16, 8>(a, p, st) : launch_norm_fwd<__nv_bfloat16, 1>(a, p, st);
    else ok = v16 ? launch_norm_fwd<float, 4>(a, p, st) : launch_norm_fwd<float, 1>(a, p, st);
    return ok ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_layer_norm_backward_workspace_size(int64_t rows, int32_t width)
{
    if (rows < 0 || width <= 0) return 0;
    return align_up(sizeof(float) * 2 * (size_t)norm_parts(rows) * width);
}

gdn_status_t gdn_layer_norm_backward(const void* x, int64_t x_stride, const void* dy, int64_t dy_stride,
                                     const void* weight, const float* mean, const float* rstd, int64_t rows,
                                     int32_t width, gdn_dtype_t in_dtype, gdn_dtype_t w_dtype, void* dx,
                                     float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                     void* stream)
{
    if (rows < 0 || rows > kMaxRows || width <= 0 || width > kMaxRows || !dtype_ok(in_dtype) || !dtype_ok(w_dtype))
        return GDN_ERR_INVALID_ARG;
    if (weight == nullptr || !aligned(weight, esize(w_dtype)) || dweight == nullptr || !aligned(dweight, 4) ||
        (dbias && !aligned(dbias, 4)))
        return GDN_ERR_INVALID_ARG;
    if (rows > 0 && (!rows_ok(x, x_stride, width, in_dtype) || !rows_ok(dy, dy_stride, width, in_dtype) ||
                     !rows_ok(dx, width, width, in_dtype) || mean == nullptr || rstd == nullptr || !aligned(mean, 4) ||
                     !aligned(rstd, 4)))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(in_dtype);
    const size_t need = gdn_layer_norm_backward_workspace_size(rows, width);
    if (overlap({{dx, rows * width, es}, {dweight, width, 4}, {dbias, width, 4}, {workspace, (int64_t)need, 1}},
                {{x, rows, x_stride, width, es}, {dy, rows, dy_stride, width, es}, {mean, rows, 4}, {rstd, rows, 4},
                 {weight, width, esize(w_dtype)}}))
        return GDN_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    gdn::NormArgs a{};
    a.x = x; a.ldx = x_stride; a.dy = dy; a.lddy = dy_stride; a.w = weight; a.w_bf16 = w_dtype == GDN_BF16;
    a.R = rows; a.D = width; a.dx = dx;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.part = static_cast<float*>(workspace);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    bool v16 = wide(x, x_stride, width, in_dtype) && wide(dy, dy_stride, width, in_dtype) &&
               wide(dx, width, width, in_dtype);
    const int vec = (int)(16 / es);
    const bool shift = !v16 && x_stride == width && dy_stride == width && aligned(x, 16) && aligned(dy, 16) &&
                       aligned(dx, 16) && width >= 4 * vec;
    v16 = v16 || shift;
    const int32_t span = shift ? width + vec - 1 : width;
    NormPlan p = v16 ? norm_plan(span, vec, 2, 256) : norm_plan(width, 1, 16, 256);
    if (p.wide && v16) p = norm_plan(span, vec, 2, 512);
    if (p.wide && v16) p = norm_plan(span, vec, 4, 512);
    p.shift = shift;
    a.tpr = p.tpr;
    int64_t parts = 0;
    if (rows > 0 && p.wide) {
        parts = std::min<int64_t>(rows, 64);
        const dim3 grid((unsigned)ceil_div(width, 256), (unsigned)parts);
        if (in_dtype == GDN_BF16) {
            gdn::k_norm_bwd_wide<__nv_bfloat16><<<(unsigned)rows, 1024, 0, st>>>(a);
            gdn::k_norm_bwd_wide_w<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
        } else {
            gdn::k_norm_bwd_wide<float><<<(unsigned)rows, 1024, 0, st>>>(a);
            gdn::k_norm_bwd_wide_w<float><<<grid, 256, 0, st>>>(a);
        }
        if (!launched()) return GDN_ERR_CUDA;
    } else if (rows > 0) {
        bool ok;
        if (in_dtype == GDN_BF16)
            ok = v16 ? launch_norm_bwd<__nv_bfloat16, 8>(a, p, &parts, st)
                     : launch_norm_bwd<__nv_bfloat16, 1>(a, p, &parts, st);
        else
            ok = v16 ? launch_norm_bwd<float, 4>(a, p, &parts, st)
                     : launch_norm_bwd<float, 1>(a, p, &parts, st);
        if (!ok) return GDN_ERR_CUDA;
    }
    const int64_t M = 2 * (int64_t)width;
    gdn::k_colsum<<<(unsigned)ceil_div(M, 32), dim3(32, 8), 0, st>>>(a.part, parts, M,
                                                                     gdn::NormGradMap{dweight, dbias, width});
    return launched() ? GDN_OK : GDN_ERR_CUDA;
}

int64_t gdn_ssm_num_chunk_states(int64_t total_tokens, int32_t num_seqs)
{
    if (total_tokens < 0 || total_tokens > kMaxRows || num_seqs < 0) return -1;
    return total_tokens / GDN_SSM_CHUNK + num_seqs;
}

size_t gdn_ssm_backward_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t channels, int32_t groups,
                                       int32_t states)
{
    if (total_tokens < 0 || num_seqs < 0 || channels <= 0 || groups <= 0 || channels % groups != 0 ||
        (states != 16 && states != 32 && states != 64))
        return 0;
    return ssm_carve(nullptr, total_tokens, num_seqs, channels, groups, states).bytes;
}

gdn_status_t gdn_ssm_forward(const gdn_ssm_t* args, const float* state_in, void* y, float* state_out,
                             float* chunk_states, int32_t* status, void* stream)
{
    const gdn_status_t bad = ssm_check(args, status, false);
    if (bad != GDN_OK) return bad;
    const gdn_ssm_t& s = *args;
    if (s.num_seqs == 0) return GDN_OK;
    if (state_out == nullptr || !aligned(state_out, 16) || (state_in && !aligned(state_in, 16)) ||
        (chunk_states && !aligned(chunk_states, 16)))
        return GDN_ERR_INVALID_ARG;
    if (s.total_tokens > 0 && !rows_ok(y, s.channels, s.channels, s.in_dtype)) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype);
    const int64_t T = s.total_tokens, per = (int64_t)s.channels * s.states, bc = (int64_t)s.groups * s.states;
    if (overlap({{y, T * s.channels, es}, {state_out, s.num_seqs * per, 4}, {status, 1, 4},
                 {chunk_states, gdn_ssm_num_chunk_states(T, s.num_seqs) * per, 4}},
                {{s.x, T, s.x_stride, s.channels, es}, {s.dt, T, s.dt_stride, s.channels, es},
                 {s.z, T, s.z_stride, s.channels, es}, {s.B, T, s.B_stride, bc, es}, {s.C, T, s.C_stride, bc, es},
                 {s.A, per, 4}, {s.D, s.channels, 4}, {s.dt_bias, s.channels, 4},
                 {s.cu_seqlens, s.num_seqs + 1LL, 4}, {state_in, s.num_seqs * per, 4}}))
        return GDN_ERR_INVALID_ARG;
    gdn::SsmArgs a = ssm_args(args, 1);  // the launch sets the channel blocks
    a.state_in = state_in; a.y = y; a.state_out = state_out; a.saved = chunk_states;
    a.status = status;
    const bool v16 = ssm_wide(args) && aligned(y, 16);
    SSM_DISPATCH(ssm_forward_launch, s.in_dtype, s.states, v16, a, static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_ssm_backward(const gdn_ssm_t* args, const void* dy, int64_t dy_stride, const float* chunk_states,
                              const float* dstate_out, void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD,
                              void* dz, float* ddt_bias, float* dstate_in, void* workspace, size_t workspace_bytes,
                              int32_t* status, void* stream)
{
    const gdn_status_t bad = ssm_check(args, status, false);
    if (bad != GDN_OK) return bad;
    const gdn_ssm_t& s = *args;
    const int64_t T = s.num_seqs > 0 ? s.total_tokens : 0;
    if (dA == nullptr || !aligned(dA, 4) || (dD && !aligned(dD, 4)) || (ddt_bias && !aligned(ddt_bias, 4)))
        return GDN_ERR_INVALID_ARG;
    if (s.num_seqs > 0 && (chunk_states == nullptr || !aligned(chunk_states, 16) || dstate_in == nullptr ||
                           !aligned(dstate_in, 16) || (dstate_out && !aligned(dstate_out, 16))))
        return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!rows_ok(dy, dy_stride, s.channels, s.in_dtype) || !rows_ok(dx, s.channels, s.channels, s.in_dtype) ||
                  !rows_ok(ddt, s.channels, s.channels, s.in_dtype) || dB == nullptr || dC == nullptr ||
                  !aligned(dB, esize(s.in_dtype)) || !aligned(dC, esize(s.in_dtype)) ||
                  (s.z != nullptr && !rows_ok(dz, s.channels, s.channels, s.in_dtype))))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype);
    const int64_t bc = (int64_t)s.groups * s.states;
    const int64_t per = (int64_t)s.channels * s.states, states = s.num_seqs * per;
    const size_t need =
        gdn_ssm_backward_workspace_size(s.total_tokens, s.num_seqs, s.channels, s.groups, s.states);
    if (overlap({{dx, T * s.channels, es}, {ddt, T * s.channels, es}, {s.z ? dz : nullptr, T * s.channels, es},
                 {dB, T * bc, es}, {dC, T * bc, es}, {dA, per, 4}, {dD, s.channels, 4}, {ddt_bias, s.channels, 4},
                 {dstate_in, states, 4}, {workspace, (int64_t)need, 1}, {status, 1, 4}},
                {{s.x, T, s.x_stride, s.channels, es}, {s.dt, T, s.dt_stride, s.channels, es},
                 {s.z, T, s.z_stride, s.channels, es}, {s.B, T, s.B_stride, bc, es}, {s.C, T, s.C_stride, bc, es},
                 {s.A, per, 4}, {s.D, s.channels, 4}, {s.dt_bias, s.channels, 4},
                 {s.cu_seqlens, s.num_seqs + 1LL, 4}, {dy, T, dy_stride, s.channels, es}, {dstate_out, states, 4},
                 {chunk_states, gdn_ssm_num_chunk_states(T, s.num_seqs) * per, 4}}))
        return GDN_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (s.num_seqs == 0) {  // no token, no state: the parameters' gradients are zero
        if (cudaMemsetAsync(dA, 0, sizeof(float) * (size_t)s.channels * s.states, st) != cudaSuccess ||
            (dD && cudaMemsetAsync(dD, 0, sizeof(float) * (size_t)s.channels, st) != cudaSuccess) ||
            (ddt_bias && cudaMemsetAsync(ddt_bias, 0, sizeof(float) * (size_t)s.channels, st) != cudaSuccess))
            return GDN_ERR_CUDA;
        return GDN_OK;
    }
    const SsmWorkspace w = ssm_carve(workspace, T, s.num_seqs, s.channels, s.groups, s.states);
    gdn::SsmBwdArgs b{};
    b.f = ssm_args(args, 2 * 128 / s.states * 4);
    b.Lc = ssm_bwd_chunk(T, s.channels, s.states);
    b.f.saved = const_cast<float*>(chunk_states);
    b.ebuf = w.ebuf; b.dsum = w.dsum; b.f.status = status;
    b.dy = dy; b.lddy = dy_stride; b.dstate_out = dstate_out;
    b.dx = dx; b.ddt = ddt; b.dz = dz; b.dstate_in = dstate_in;
    b.partA = w.partA; b.partD = w.partD; b.partBC = w.partBC;
    const bool v16 = ssm_wide(args) && wide(dy, dy_stride, b.f.Dg, s.in_dtype) && aligned(dx, 16) && aligned(ddt, 16) &&
                     (s.z == nullptr || aligned(dz, 16));
    SSM_DISPATCH(ssm_backward_launch, s.in_dtype, s.states, v16, b, dB, dC, dA, dD, ddt_bias, st);
}

gdn_status_t gdn_ssm_step(const gdn_ssm_t* args, const float* state, float* state_out, void* y, void* stream)
{
    const gdn_status_t bad = ssm_check(args, nullptr, true);
    if (bad != GDN_OK) return bad;
    const gdn_ssm_t& s = *args;
    if (s.num_seqs == 0) return GDN_OK;
    if (state == nullptr || state_out == nullptr || !aligned(state, 16) || !aligned(state_out, 16) ||
        !rows_ok(y, s.channels, s.channels, s.in_dtype))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(s.in_dtype);
    const int64_t N = s.num_seqs, per = (int64_t)s.channels * s.states;
    const int64_t bc = (int64_t)s.groups * s.states;
    if (overlap({{y, N * s.channels, es}, {state_out, N * per, 4}},
                {{s.x, N, s.x_stride, s.channels, es}, {s.dt, N, s.dt_stride, s.channels, es},
                 {s.z, N, s.z_stride, s.channels, es}, {s.B, N, s.B_stride, bc, es}, {s.C, N, s.C_stride, bc, es},
                 {s.A, per, 4}, {s.D, s.channels, 4}, {s.dt_bias, s.channels, 4},
                 {state != state_out ? state : nullptr, N * per, 4}}))
        return GDN_ERR_INVALID_ARG;
    gdn::SsmArgs a = ssm_args(args, 1);
    a.state_in = state; a.state_out = state_out; a.y = y;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (s.in_dtype == GDN_BF16) {
        if (s.states == 16) return ssm_step_launch<__nv_bfloat16, 16>(a, st);
        if (s.states == 32) return ssm_step_launch<__nv_bfloat16, 32>(a, st);
        return ssm_step_launch<__nv_bfloat16, 64>(a, st);
    }
    if (s.states == 16) return ssm_step_launch<float, 16>(a, st);
    if (s.states == 32) return ssm_step_launch<float, 32>(a, st);
    return ssm_step_launch<float, 64>(a, st);
}

}  // extern "C"

// glu_ops.cu -- host side of the gated feed-forward block (gdn_cpr.h).
//
// As layer_ops.cu: it validates on the host, carves the caller's workspace and
// enqueues on the caller's stream; it allocates nothing, keeps no state and
// never synchronises.
#include "layer_host.cuh"
#include "tensor_map.cuh"
#include "k_glu.cuh"

namespace {

using bf16 = __nv_bfloat16;

// Tensor map of a [rows, cols] bf16 matrix, rows ld elements apart, for boxes of 64 columns with 128-byte swizzle.  Boxes
// that reach past the end are filled with zeros.
bool matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix that TMA can read: whole 16-byte rows at a 16-byte address.
bool tma_rows(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }
int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }

// x and the weights, or their aligned copies in the workspace
struct GluOperands {
    const void *x, *wg, *wu;
    int64_t ldx, ldg, ldu;
    size_t bytes;  // of the copies
};

// Carves the copies from p (which may be null: sizes only).
GluOperands glu_operands(const gdn_glu_t& s, unsigned char* p)
{
    GluOperands o{s.x, s.w_gate, s.w_up, s.x_stride, s.gate_stride, s.up_stride, 0};
    const int64_t ld = pad8(s.width);
    auto copy = [&](const void*& q, int64_t& l, int64_t rows) {
        if (rows == 0 || tma_rows(q, l)) return;
        q = p + o.bytes;
        l = ld;
        o.bytes += align_up((size_t)rows * ld * 2);
    };
    copy(o.x, o.ldx, s.rows);
    copy(o.wg, o.ldg, s.inner);
    copy(o.wu, o.ldu, s.inner);
    return o;
}

bool glu_align(const gdn_glu_t& s, const GluOperands& o, int sms, cudaStream_t st)
{
    gdn::GluAlign a{};
    a.cols = s.width;
    a.ldd = pad8(s.width);
    int m = 0;
    int64_t most = 0;
    auto add = [&](const void* src, int64_t lds, const void* dst, int64_t rows) {
        if (src == dst || rows == 0) return;
        a.src[m] = static_cast<const uint16_t*>(src);
        a.dst[m] = static_cast<uint16_t*>(const_cast<void*>(dst));
        a.lds[m] = lds;
        a.rows[m++] = rows;
        most = std::max(most, rows);
    };
    add(s.x, s.x_stride, o.x, s.rows);
    add(s.w_gate, s.gate_stride, o.wg, s.inner);
    add(s.w_up, s.up_stride, o.wu, s.inner);
    if (m == 0) return true;
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(most * (a.ldd / 8), 256), (int64_t)sms * 8), (unsigned)m);
    gdn::k_glu_align<<<grid, 256, 0, st>>>(a);
    return launched();
}

gdn_status_t glu_check(const gdn_glu_t* s, const int32_t* status)
{
    if (s == nullptr || s->rows < 0 || s->rows > kMaxRows || s->width <= 0 || s->inner <= 0 || s->width > kMaxRows ||
        s->inner > kMaxRows || !dtype_ok(s->in_dtype) || (s->act != GDN_ACT_SILU && s->act != GDN_ACT_GELU) ||
        !aligned(status, 4))
        return GDN_ERR_INVALID_ARG;
    if (s->in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (!rows_ok(s->w_gate, s->gate_stride, s->width, s->in_dtype) || !rows_ok(s->w_up, s->up_stride, s->width, s->in_dtype))
        return GDN_ERR_INVALID_ARG;
    if (s->rows > 0 && !rows_ok(s->x, s->x_stride, s->width, s->in_dtype)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Before the product's maps are made
template <int MODE, bool SAVE = false, int ACT = gdn::kGluSilu>
bool glu_ready()
{
    return raise_smem<gdn::glu_gemm_smem(SAVE)>(gdn::k_glu_gemm<MODE, SAVE, ACT>);
}

template <int MODE, bool SAVE = false, int ACT = gdn::kGluSilu>
gdn_status_t glu_gemm(gdn::GluMaps& maps, gdn::GluGemmArgs& a, int sms, cudaStream_t st)
{
    a.tiles_m = (int32_t)ceil_div(a.M, 256);
    a.tiles_n = (int32_t)ceil_div(a.N, MODE == gdn::kGluFwd ? 128 : 256);
    a.tiles = (int64_t)a.tiles_m * a.tiles_n * a.problems * a.splits;
    const unsigned pairs = (unsigned)std::min<int64_t>(a.tiles, std::max(1, sms / 2));
    return launch_next(gdn::k_glu_gemm<MODE, SAVE, ACT>, dim3(2 * pairs), dim3(gdn::kGluGemmThreads), gdn::glu_gemm_smem(SAVE), 0, st, maps, a)
               ? GDN_OK : GDN_ERR_CUDA;
}

// Whether the weights are streamed past the tokens: up to 128 tokens, and where the pairs of SMs would have at most 16 tiles, or 32
// for up to 256 tokens, whose results leave room for one block per SM only (300 x 4096 x 1024 18 us, in tiles 27; 1024 x 2048 x 512 15
// and 17; with 32 tiles, 1024 x 1024 x 1024, 17 and 13.  Behind an L2 full of written lines: 256 x 4096 x 4096 37 and 39, x 6144
// 49 and 43, x 28672 160 and 125; 128 x 4096 x 8192 43 and 47).
bool glu_is_few(int64_t rows, int64_t inner)
{
    return rows <= 128 || ceil_div(rows, 256) * ceil_div(inner, 128) <= (rows <= 256 ? 32 : 16);
}

constexpr int64_t kStageK = 2 * gdn::kGluK;  // k of a stage of the pair's product

// Tensor map of an operand of the pair's product: boxes of 64 columns by 128 rows, or (wide: whole 64 columns) of two such runs
// side by side.
bool operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, bool wide_boxes)
{
    if (!wide_boxes) return matrix_map(map, base, rows, cols, ld, 128);
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
    const cuuint32_t box[3] = {64u, 128u, 2u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Parts of the K axis of a product with few tiles: enough for every pair of SMs, each of at least 4 stages.
int glu_splits(int64_t tiles, int64_t ksteps, int sms)
{
    const int64_t want = std::max<int64_t>(1, (sms / 2) / tiles);
    return (int)std::max<int64_t>(1, std::min<int64_t>({want, ksteps / 4, 64}));
}

// Blocks take equal shares of the units, in multiples of 8 up to 64: one block per SM, with all of its shared memory, where 64 units
// for each SM are enough, or two, or three where all blocks then run at once (behind an L2 full of written lines: 100 x 4096 x 20480
// 82 us with three, 117 with two; 28672, a block too many for three, 176 and 125).  With fewer units than 32 for each SM, clusters of
// 2 or 4 blocks share the K axis.  A stage holds 4, 2 or 1 times 64 columns, so that there are at least three where there is
// room (100 x 4096 x 11008 55 us, with one stage 72; 1 x 4096 x 28672 94 and 104).
template <int NB>
gdn_status_t glu_few(const GluOperands& o, const gdn_glu_t& s, gdn::GluFewArgs& a, int sms, cudaStream_t st)
{
    // a cluster's blocks lie in one group of SMs, of which a few are left over: a full house would come in two waves
    const int groups = (int)ceil_div(s.rows, NB);  // of tokens
    const auto slots = [&](int S) { return std::max(1, (S > 1 ? sms * 7 / 8 : sms) / groups); };
    int S = 1;
    while (S < 4 && ceil_div((int64_t)s.inner * S * 2, slots(2)) <= 64 && a.ksteps >= 8 * S) S *= 2;
    const int64_t per = ceil_div((int64_t)s.inner * S, slots(S));  // units of an SM
    const int resident = per <= 64 ? 1 : per <= 128 || per > 192 ? 2 : 3;
    a.rows = (int)std::min<int64_t>(64, ceil_div(ceil_div((int64_t)s.inner * S, (int64_t)slots(S) * resident), 8) * 8);
    const size_t room = (size_t)(resident == 1 ? 224 : resident == 2 ? 110 : 72) * 1024 - gdn::kGluHalf, chunk = gdn::glu_few_chunk(NB, a.rows);
    a.chunks = NB > 128 ? 1 : NB > 16 ? 2 : 4;
    while (a.chunks > 1 && room / (a.chunks * chunk) < 3) a.chunks /= 2;
    a.stages = (int)std::min<size_t>(gdn::kGluFewStages, room / (a.chunks * chunk));
    const size_t smem = gdn::glu_few_tiles(NB, a.rows, a.stages, a.chunks) + 1024 + 512;
    auto k = s.act == GDN_ACT_SILU ? gdn::k_glu_few<NB, gdn::kGluSilu> : gdn::k_glu_few<NB, gdn::kGluGelu>;
    if (!raise_smem(k, smem)) return GDN_ERR_CUDA;
    gdn::GluFewMaps maps;
    if (!matrix_map(&maps.x, o.x, s.rows, s.width, o.ldx, NB) || !matrix_map(&maps.wg, o.wg, s.inner, s.width, o.ldg, a.rows) ||
        !matrix_map(&maps.wu, o.wu, s.inner, s.width, o.ldu, a.rows))
        return GDN_ERR_CUDA;
    const dim3 grid((unsigned)ceil_div(s.inner, a.rows) * S, (unsigned)ceil_div(s.rows, NB));
    return launch_next(k, grid, dim3(gdn::kGluThreads), smem, S, st, maps, a) ? GDN_OK : GDN_ERR_CUDA;
}

// The backward's workspace: dg and du, rows ld apart; aligned copies; the splits' partial products.
struct GluBackwardPlan {
    int64_t ld, grad_rows;  // rows of dg and du: with those of what their rounding left, twice the tokens
    int splits_x, splits_w;
    size_t copies, part, bytes;  // offsets
};

GluBackwardPlan glu_backward_plan(const gdn_glu_t& s, int sms)
{
    GluBackwardPlan p;
    p.ld = pad8(s.inner);
    p.grad_rows = s.rows <= 128 ? 2 * s.rows : s.rows;
    const int64_t tx = ceil_div(s.rows, 256) * ceil_div(s.width, 256);
    const int64_t tw = 2 * ceil_div(s.inner, 256) * ceil_div(s.width, 256);
    p.splits_x = s.rows > 0 ? glu_splits(tx, 2 * ceil_div(s.inner, kStageK), sms) : 1;
    p.splits_w = s.rows > 0 ? glu_splits(tw, ceil_div(s.rows, kStageK), sms) : 1;
    p.copies = 2 * align_up((size_t)p.grad_rows * p.ld * 2);
    p.part = p.copies + glu_operands(s, nullptr).bytes;
    const bool joined = p.splits_x > 1 || p.grad_rows > s.rows;
    const size_t px = joined ? sizeof(float) * (size_t)p.splits_x * p.grad_rows * s.width : 0;
    const size_t pw = p.splits_w > 1 ? sizeof(float) * 2 * (size_t)p.splits_w * s.inner * s.width : 0;
    p.bytes = p.part + align_up(std::max(px, pw));
    return p;
}

template <bool LO>
auto glu_grad(int32_t act, bool whole)
{
    return act == GDN_ACT_SILU ? (whole ? gdn::k_glu_grad<true, gdn::kGluSilu, LO> : gdn::k_glu_grad<false, gdn::kGluSilu, LO>)
                               : (whole ? gdn::k_glu_grad<true, gdn::kGluGelu, LO> : gdn::k_glu_grad<false, gdn::kGluGelu, LO>);
}

template <typename OT>
bool glu_join(const float* part, int splits, int64_t n, void* o0, void* o1, int problems, int sms, cudaStream_t st)
{
    return launch_next(gdn::k_glu_join<OT>, dim3((unsigned)std::min<int64_t>(ceil_div(n * problems, 256), (int64_t)sms * 16)), dim3(256), 0, 0, st,
                       part, splits, n, static_cast<OT*>(o0), static_cast<OT*>(o1), problems);
}

}  // namespace

extern "C" {

int64_t gdn_glu_saved_size(int64_t rows, int32_t inner)
{
    return rows < 0 || inner <= 0 ? -1 : 6 * rows * (int64_t)inner;
}

size_t gdn_glu_forward_workspace_size(const gdn_glu_t* args)
{
    return glu_check(args, nullptr) == GDN_OK ? glu_operands(*args, nullptr).bytes : 0;
}

gdn_status_t gdn_glu_forward(const gdn_glu_t* args, void* h, void* saved, void* workspace, size_t workspace_bytes,
                             int32_t* status, void* stream)
{
    const gdn_status_t bad = glu_check(args, status);
    if (bad != GDN_OK) return bad;
    const gdn_glu_t& s = *args;
    if (s.rows == 0) return GDN_OK;
    if (!rows_ok(h, s.inner, s.inner, s.in_dtype) || !aligned(saved, 16)) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_glu_forward_workspace_size(args);
    const int64_t R = s.rows, F = s.inner, D = s.width;
    if (overlap({{h, R * F, 2}, {saved, gdn_glu_saved_size(R, s.inner), 1}, {workspace, (int64_t)need, 1}, {status, 1, 4}},
                {{s.x, R, s.x_stride, D, 2}, {s.w_gate, F, s.gate_stride, D, 2}, {s.w_up, F, s.up_stride, D, 2}}))
        return GDN_ERR_INVALID_ARG;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return GDN_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const GluOperands o = glu_operands(s, static_cast<unsigned char*>(workspace));
    if (!glu_align(s, o, sms, st)) return GDN_ERR_CUDA;
    const int32_t ksteps = (int32_t)ceil_div(D, gdn::kGluK);
    if (glu_is_few(R, F)) {
        gdn::GluFewArgs a{};
        a.T = (int32_t)R; a.F = s.inner; a.ksteps = ksteps; a.h = h; a.saved = static_cast<uint16_t*>(saved); a.status = status;
        if (R <= 16) return glu_few<16>(o, s, a, sms, st);
        if (R <= 32) return glu_few<32>(o, s, a, sms, st);
        if (R <= 64) return glu_few<64>(o, s, a, sms, st);
        if (R <= 128) return glu_few<128>(o, s, a, sms, st);
        return glu_few<256>(o, s, a, sms, st);
    }
    const bool silu = s.act == GDN_ACT_SILU;
    if (!(silu ? (saved ? glu_ready<gdn::kGluFwd, true, gdn::kGluSilu>() : glu_ready<gdn::kGluFwd, false, gdn::kGluSilu>())
               : (saved ? glu_ready<gdn::kGluFwd, true, gdn::kGluGelu>() : glu_ready<gdn::kGluFwd, false, gdn::kGluGelu>())))
        return GDN_ERR_CUDA;
    gdn::GluMaps maps;
    const bool wide_boxes = D % 64 == 0;
    if (!operand_map(&maps.a[0], o.x, R, D, o.ldx, wide_boxes) || !operand_map(&maps.b[0], o.wg, F, D, o.ldg, wide_boxes) ||
        !operand_map(&maps.b[1], o.wu, F, D, o.ldu, wide_boxes))
        return GDN_ERR_CUDA;
    maps.a[1] = maps.a[0];
    gdn::GluGemmArgs a{};
    a.M = R; a.N = F; a.ksteps = (int32_t)ceil_div(D, kStageK); a.parts = 1; a.problems = 1; a.splits = 1; a.wide = wide_boxes;
    a.out[0] = h;
    a.saved = static_cast<uint16_t*>(saved); a.status = status;
    if (silu)
        return saved ? glu_gemm<gdn::kGluFwd, true, gdn::kGluSilu>(maps, a, sms, st)
                     : glu_gemm<gdn::kGluFwd, false, gdn::kGluSilu>(maps, a, sms, st);
    return saved ? glu_gemm<gdn::kGluFwd, true, gdn::kGluGelu>(maps, a, sms, st)
                 : glu_gemm<gdn::kGluFwd, false, gdn::kGluGelu>(maps, a, sms, st);
}

size_t gdn_glu_backward_workspace_size(const gdn_glu_t* args)
{
    const int sms = sm_count();
    return glu_check(args, nullptr) == GDN_OK && sms > 0 ? glu_backward_plan(*args, sms).bytes : 0;
}

gdn_status_t gdn_glu_backward(const gdn_glu_t* args, const void* dh, int64_t dh_stride, const void* saved, void* dx,
                              void* dw_gate, void* dw_up, gdn_dtype_t dw_dtype, void* workspace, size_t workspace_bytes,
                              int32_t* status, void* stream)
{
    const gdn_status_t bad = glu_check(args, status);
    if (bad != GDN_OK) return bad;
    const gdn_glu_t& s = *args;
    const int64_t R = s.rows, F = s.inner, D = s.width;
    if (!dtype_ok(dw_dtype)) return GDN_ERR_INVALID_ARG;
    const size_t ws = esize(dw_dtype);
    if (dw_gate == nullptr || dw_up == nullptr || !aligned(dw_gate, ws) || !aligned(dw_up, ws)) return GDN_ERR_INVALID_ARG;
    if (R > 0 && (!rows_ok(dh, dh_stride, F, s.in_dtype) || !rows_ok(dx, D, D, s.in_dtype) || saved == nullptr ||
                  !aligned(saved, 16)))
        return GDN_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto shared = [&](const void* w, size_t n) {
        return overlap({{R > 0 ? dx : nullptr, R * D, 2}, {dw_gate, F * D, ws}, {dw_up, F * D, ws}, {w, (int64_t)n, 1}, {status, 1, 4}},
                       {{s.x, R, s.x_stride, D, 2}, {s.w_gate, F, s.gate_stride, D, 2}, {s.w_up, F, s.up_stride, D, 2},
                        {dh, R, dh_stride, F, 2}, {saved, gdn_glu_saved_size(R, s.inner), 1}});
    };
    if (shared(nullptr, 0)) return GDN_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return GDN_ERR_CUDA;
    const GluBackwardPlan p = glu_backward_plan(s, sms);
    if (R > 0 && shared(workspace, p.bytes)) return GDN_ERR_INVALID_ARG;
    if (R == 0)  // no token: the weights' gradients are zero
        return cudaMemsetAsync(dw_gate, 0, ws * (size_t)F * D, st) == cudaSuccess &&
                       cudaMemsetAsync(dw_up, 0, ws * (size_t)F * D, st) == cudaSuccess
                   ? GDN_OK : GDN_ERR_CUDA;
    if (workspace == nullptr || workspace_bytes < p.bytes) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    unsigned char* base = static_cast<unsigned char*>(workspace);
    bf16 *dg = reinterpret_cast<bf16*>(base), *du = reinterpret_cast<bf16*>(base + p.copies / 2);
    float* part = reinterpret_cast<float*>(base + p.part);
    const GluOperands o = glu_operands(s, base + p.copies);
    if (!glu_align(s, o, sms, st)) return GDN_ERR_CUDA;

    const unsigned blocks = (unsigned)std::min<int64_t>(ceil_div(R * (p.ld / 8), 256), (int64_t)sms * 32);
    const uint16_t *g = static_cast<const uint16_t*>(dh), *sv = static_cast<const uint16_t*>(saved);
    const bool whole = F % 8 == 0 && wide(dh, dh_stride, F, s.in_dtype);
    const bool few = p.grad_rows > R;
    auto k = few ? glu_grad<true>(s.act, whole) : glu_grad<false>(s.act, whole);
    if (!launch_next(k, dim3(blocks), dim3(256), 0, 0, st, g, dh_stride, sv, R, F, dg, du, p.ld)) return GDN_ERR_CUDA;

    if (!glu_ready<gdn::kGluDx>() || !glu_ready<gdn::kGluDw>()) return GDN_ERR_CUDA;
    gdn::GluMaps mx, mw;
    const bool wide_boxes = D % 64 == 0 && F % 64 == 0;
    if (!operand_map(&mx.a[0], dg, p.grad_rows, F, p.ld, wide_boxes) || !operand_map(&mx.a[1], du, p.grad_rows, F, p.ld, wide_boxes) ||
        !operand_map(&mx.b[0], o.wg, F, D, o.ldg, wide_boxes) || !operand_map(&mx.b[1], o.wu, F, D, o.ldu, wide_boxes) ||
        !operand_map(&mw.b[0], o.x, R, D, o.ldx, wide_boxes))
        return GDN_ERR_CUDA;
    mw.a[0] = mx.a[0]; mw.a[1] = mx.a[1]; mw.b[1] = mw.b[0];
    gdn::GluGemmArgs a{};
    a.wide = wide_boxes;
    a.M = p.grad_rows; a.N = D; a.ksteps = (int32_t)ceil_div(F, kStageK); a.parts = 2; a.problems = 1; a.splits = p.splits_x;
    const int sums = few ? 2 * p.splits_x : p.splits_x;  // [splits][grad_rows][D]
    a.out[0] = dx; a.partial = sums > 1 ? part : nullptr; a.status = status;
    gdn_status_t r = glu_gemm<gdn::kGluDx>(mx, a, sms, st);
    if (r != GDN_OK) return r;
    if (sums > 1 && !glu_join<bf16>(part, sums, R * D, dx, nullptr, 1, sms, st)) return GDN_ERR_CUDA;
    a.M = F; a.N = D; a.ksteps = (int32_t)ceil_div(R, kStageK); a.parts = few ? 2 : 1; a.problems = 2; a.splits = p.splits_w;
    a.lo = (int32_t)R; a.partial = p.splits_w > 1 ? part : nullptr;
    a.out[0] = dw_gate; a.out[1] = dw_up; a.out_f32 = dw_dtype == GDN_F32;
    r = glu_gemm<gdn::kGluDw>(mw, a, sms, st);
    if (r != GDN_OK) return r;
    if (p.splits_w > 1) {
        const bool ok = dw_dtype == GDN_F32 ? glu_join<float>(part, p.splits_w, F * D, dw_gate, dw_up, 2, sms, st)
                                            : glu_join<bf16>(part, p.splits_w, F * D, dw_gate, dw_up, 2, sms, st);
        if (!ok) return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

}  // extern "C"

// k_glu.cuh -- the gated feed-forward block's projections, activation and product, forward and backward, on the
// 5th-generation tensor cores (sm_100a).
//
//     g = x Wg^T,  u = x Wu^T,  h = act(g) u
//     dg = dh u act'(g),  du = dh act(g)
//     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// k_glu_gemm is the product of all three: a pair of CTAs on neighbouring SMs makes a tile of 256 x 256
// with tcgen05.mma.cta_group::2 (bf16 operands, fp32 accumulators in tensor memory), so that each SM fetches
// half of either operand: 32 KB per 128 x 256 x 64 products, 64 bytes per cycle at the
// tensor cores' rate.  TMA fills a ring of shared memory stages, one thread issues the products, and eight
// warps empty one accumulator (256 of 512 columns) while the next tile fills the other.
//   forward   A = x, B = 128 rows of Wg (from the first CTA) and the same rows of Wu (from the second): a row of the
//             accumulator holds g and u of the same 128 units, so act(g) u is made where it is read
//   dx        A = dg, then du; B = Wg, then Wu, with the output's columns contiguous (read as K x N)
//   dW        A = dg or du as K x M, B = x as K x N; the two gradients are the two halves of the tiles
// dg and du are rounded to bf16, which adds to the gradients about what the rounding of a bf16 result adds: their error is 1.41 to 1.45
// times that of a result rounded once, from 129 to 4096 tokens alike (72 x 80 and 512 x 1024), and 1.7e-3 of the norm in the
// weights' gradients in fp32 (bf16 results: 2.3e-3).  Up to 128 tokens, where a few of them can dominate (2.2 at 1 x 72 x 80), what
// the rounding left goes through the products as well, 1.00 and 1e-5, in room that the tiles have anyway: as more rows of dx, of
// which a tile has 256, joined with the splits of K, and as more rows of K for dW, of which a stage has 128.  Beyond it would double the
// tiles.
//
// k_glu_few serves few tokens, where the weights' bytes bound it: a block holds up to 64 rows of Wg and the same ones of Wu
// as the M side of one product, as many as give every SM the same share of them, and streams them past the
// tokens (the N side, 16 to 256).  Where that would leave few rows, a cluster of blocks shares the K axis,
// and its partial sums meet in distributed shared memory, in a fixed order.
//
// Bound by the tensor cores: 8192 x 4096 x 8192 takes the forward 655 us (1679 TFLOP/s; 708 with what the backward reads), dx
// 680 (1617) and the weights' gradients 712 us (1544); a second under load, with the clock held down by the power limit, about
// 1300.  k_glu_grad between them 123 us.  64 x 4096 x 8192 takes k_glu_few 27 us, 1 x 2048 x 8192 15 us (5.0 and 4.5 TB/s).
#pragma once

#include "cluster.cuh"
#include "k_tc.cuh"
#include "layer_common.cuh"
#include "tma.cuh"

namespace gdn {

constexpr int kGluSilu = 0, kGluGelu = 1;

// ------------------------------------------------------------- the activation
// act(g) and act'(g).  gelu: 0.5 g (1 + tanh t) = g sigmoid(2 t), 2 t = sqrt(8 / pi) (g + 0.044715 g^3)
// (ACT is a template's: a branch for each element would keep them from overlapping.)
template <int ACT>
__device__ __forceinline__ float glu_act(float g)
{
    if constexpr (ACT == kGluSilu) return silu(g);
    const float t = 1.5957691216057308f * __fmaf_rn(0.044715f * g * g, g, g);
    return g * sigmoid(t);
}
template <int ACT>
__device__ __forceinline__ void glu_act2(float g, float& a, float& slope)
{
    if constexpr (ACT == kGluSilu) {
        const float s = sigmoid(g);
        a = g * s;
        slope = s * __fmaf_rn(g, 1.0f - s, 1.0f);
    } else {
        // a square that overflowed would make the slope of the far ends 0 times infinity
        const float g2 = fminf(g * g, 1e30f), s = sigmoid(1.5957691216057308f * __fmaf_rn(0.044715f * g2, g, g));
        a = g * s;
        slope = __fmaf_rn(a * (1.0f - s), 1.5957691216057308f * __fmaf_rn(0.134145f, g2, 1.0f), s);
    }
}

// What the backward reads of the forward: g and u to 24 bits (15 of mantissa), as planes of 16-bit words
// [3][rows][inner]: their upper halves, and the next bytes of both in one word.  In bf16 alone the
// rounding of g and u would add to dg, du and the weights' gradients as much again as the rounding of the
// products' operands; 24 bits leave about 2^-16, for 6 bytes in place of 4 (fp32: 8): cut off here, which takes 2^-16
// ln 2 of a value on average, and given that back when they are read, so that nothing is drawn towards zero (1.35 2^-16 at most; 0 and
// infinities stay what they are).  (Rounded here, the products of few columns waited for their epilogue: 20110 x
// 128 x 11712 610 us in place of 498.)
__device__ __forceinline__ void glu_pack(float g, float u, uint16_t& gh, uint16_t& uh, uint16_t& low)
{
    const uint32_t a = __float_as_uint(g), b = __float_as_uint(u);
    gh = (uint16_t)(a >> 16);
    uh = (uint16_t)(b >> 16);
    low = (uint16_t)(((a >> 8) & 0xff) | (b & 0xff00));
}
__device__ __forceinline__ void glu_unpack(uint16_t gh, uint16_t uh, uint16_t low, float& g, float& u)
{
    constexpr float back = 1.0000106096f;  // 1 + 2^-16 ln 2
    g = __uint_as_float(((uint32_t)gh << 16) | ((uint32_t)(low & 0xff) << 8)) * back;
    u = __uint_as_float(((uint32_t)uh << 16) | (low & 0xff00u)) * back;
}

// ------------------------------------------------------------- primitives
// A tile of a matrix into this CTA's shared memory; its bytes count on the barrier at cluster address `mbar`, which
// may be the pair's other CTA's.
__device__ __forceinline__ void tma_pair_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t mbar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
        : "memory");
}
// The same of 64 columns, a second run of them, and rows in between: two boxes of a matrix side by side
__device__ __forceinline__ void tma_pair_3d(void* dst, const CUtensorMap* map, int y, int chunk, uint32_t mbar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(chunk), "r"(mbar)
        : "memory");
}
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* mbar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(mbar))
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
template <int GROUP>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if constexpr (GROUP == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// One arrival at the barrier of both CTAs of the pair when every product issued before is complete.
__device__ __forceinline__ void mma_commit_pair(uint64_t* mbar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(mbar)), "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, float (&x)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Operand tiles lie as TMA leaves them with 128-byte swizzle.  K-major: rows of 64 k; the next 8 rows are
// 1024 bytes on.  Otherwise (k by k rows of 64 columns): the next 8 k are 1024 bytes on, the next 64
// columns a box on.
constexpr int kGluK = 64;  // k of a box of a K-major operand
// `box`: the bytes of 64 columns by the stage's k, for operands that are not K-major
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, bool kmajor, uint32_t box = 0)
{
    const uint64_t lbo = kmajor ? 1 : box >> 4, sbo = 1024 >> 4;
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (lbo << 16) | (sbo << 32) | (1ull << 46) | (2ull << 61);
}
// fp32 accumulators, bf16 operands
__host__ __device__ constexpr uint32_t bf16_idesc(int m, int n, bool a_kmajor, bool b_kmajor)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_kmajor ? 0u : 1u) << 15) | ((b_kmajor ? 0u : 1u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ------------------------------------------------------------- the pair's product
enum GluMode { kGluFwd = 0, kGluDx = 1, kGluDw = 2 };

struct GluMaps {
    CUtensorMap a[2], b[2];
};

struct GluGemmArgs {
    int64_t M, N;        // of the output (forward: tokens and units)
    int32_t ksteps;      // stages of one part of K
    int32_t wide;        // the maps' boxes are whole operands of a stage: rows of whole 64 columns
    int32_t parts;       // dx: 2 (dg, then du); dW of few tokens: 2 (dg or du, then what its rounding left, `lo` rows on)
    int32_t lo;
    int32_t tiles_m, tiles_n, problems, splits;
    int64_t tiles;       // tiles_m tiles_n problems splits
    void* out[2];
    uint16_t* saved;     // forward: planes [3][M][N], or null
    float* partial;      // [problems][splits][M][N], to be joined, or null
    int32_t out_f32;
    int32_t* status;
};

struct GluTile {
    int64_t m, n;  // first row (of the pair) and first column
    int problem, split, k0, k1;
};

// A stage holds 128 k of either operand.  The larger the boxes that fetch it the better: 8192 x 4096 x 8192 takes the
// forward 792 us with boxes of 8 KB, 705 with 16 KB and 674 with 32 KB (655 since), the weights' gradients 829, 735 and 712.
constexpr uint32_t kGluHalf = 128 * kGluK * 2;     // 128 rows by 64 k, or 64 columns by 128 k
constexpr uint32_t kGluOperand = 2 * kGluHalf;     // bytes of one operand of one CTA in a stage
constexpr int kGluStages = 3;
constexpr int kGluThreads = 256;                   // of k_glu_few
constexpr int kGluOutWarps = 8, kGluGemmThreads = 128 + 32 * kGluOutWarps;
__host__ __device__ constexpr uint32_t glu_staging(bool save) { return kGluOutWarps * (save ? 2 : 1) * 2048; }
__host__ __device__ constexpr size_t glu_gemm_smem(bool save)
{
    return (size_t)kGluStages * 2 * kGluOperand + glu_staging(save) + 1024 + 256;
}

// Tiles in groups of 8 or 16 rows of tiles, down the rows first: what is on the chip at a time shares few rows and columns.
// The forward by 16: 16384 x 2048 x 8192 takes 668 us and by 8 688 (8192 x 4096 x 8192: 655 and 673; only few K with what the
// backward reads lose, 32768 x 1024 x 2048 218 and 213); dx of the first 687 and 679, the weights' gradients 716 and 712.
template <int MODE>
__device__ __forceinline__ GluTile glu_tile(const GluGemmArgs& a, int64_t id)
{
    GluTile t;
    const int64_t per = (int64_t)a.tiles_m * a.tiles_n;
    const int64_t ps = id / per;
    int64_t i = id - ps * per;
    t.problem = (int)(ps / a.splits);
    t.split = (int)(ps - (int64_t)t.problem * a.splits);
    constexpr int64_t GROUP = MODE == kGluFwd ? 16 : 8;
    const int64_t group = i / (GROUP * a.tiles_n);
    const int64_t rows = min(GROUP, a.tiles_m - group * GROUP);
    i -= group * GROUP * a.tiles_n;
    t.m = (group * GROUP + i % rows) * 256;
    t.n = (i / rows) * (MODE == kGluFwd ? 128 : 256);
    const int64_t all = (int64_t)a.ksteps * a.parts;
    t.k0 = (int)(all * t.split / a.splits);
    t.k1 = (int)(all * (t.split + 1) / a.splits);
    return t;
}

// A warp's 32 rows of 64 bytes on their way to memory, where a row lies across threads: each thread puts its row's 16-byte
// pieces, then the warp stores whole rows of them, eight at a time.  Straight from the threads' rows every store would
// touch 32 lines, which bound the products of few columns (20110 x 128 x 11712 with what the backward
// reads: 1138 us).
__device__ __forceinline__ uint4* glu_piece(unsigned char* st, int row, int piece)
{
    return reinterpret_cast<uint4*>(st + row * 64 + ((piece ^ (row >> 1)) & 3) * 16);  // no two of 8 threads in one bank
}
// `bytes` of the first `rows` rows to `to`, ld bytes apart.  Rows of odd widths start anywhere: 16 bytes of memory then begin in
// one piece and end in the next, and of a row's 64 bytes the 16 at its ends go in twos.
__device__ __forceinline__ void glu_rows_out(unsigned char* st, unsigned char* to, int64_t ld, int rows, int bytes, int lane)
{
    const uintptr_t any = reinterpret_cast<uintptr_t>(to) | (uintptr_t)ld | (uintptr_t)bytes;
    if ((any & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), p = lane & 3;
            if (r < rows && p * 16 < bytes) *reinterpret_cast<uint4*>(to + r * ld + p * 16) = *glu_piece(st, r, p);
        }
    } else if (bytes == 64) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int at = i * 32 + lane, r = at / 3, k = at - r * 3 + 1;
            unsigned char* row = to + r * ld;
            const int s = (int)(reinterpret_cast<uintptr_t>(row) & 15);
            const uint4 v = *glu_piece(st, r, k);
            if (r < rows) *reinterpret_cast<uint4*>(row + 16 * k - s) = s == 0 ? v : bytes_at(*glu_piece(st, r, k - 1), v, 16 - s);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), j = lane & 7;
            uint16_t* row = reinterpret_cast<uint16_t*>(to + r * ld);
            const int s = (int)(reinterpret_cast<uintptr_t>(row) & 15), e = 2 * j < 16 - s ? j : 24 + j;
            if (r < rows) row[e] = reinterpret_cast<const uint16_t*>(glu_piece(st, r, e >> 3))[e & 7];
        }
    } else {
#pragma unroll 4
        for (int r = 0; r < 32; ++r)
            if (r < rows && lane * 2 < bytes)
                *reinterpret_cast<uint16_t*>(to + r * ld + lane * 2) = reinterpret_cast<const uint16_t*>(glu_piece(st, r, lane >> 3))[lane & 7];
    }
}

// SAVE: the forward leaves what the backward reads.
template <int MODE, bool SAVE, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGluGemmThreads, 1)
    k_glu_gemm(const __grid_constant__ GluMaps maps, const GluGemmArgs a)
{
    constexpr bool AK = MODE != kGluDw, BK = MODE == kGluFwd;  // which operands are K-major
    constexpr int ST = kGluStages;
    constexpr uint32_t IDESC = bf16_idesc(256, 256, AK, BK);
    extern __shared__ unsigned char glu_smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(glu_smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char* staging = smem + ST * 2 * kGluOperand;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + glu_staging(SAVE));  // [ST] used in the first CTA
    uint64_t* empty = full + ST;      // [ST] one per CTA
    uint64_t* done = empty + ST;      // [2] the accumulators are complete
    uint64_t* drained = done + 2;     // [2] used in the first CTA: both CTAs have read an accumulator
    uint32_t* slot = reinterpret_cast<uint32_t*>(drained + 2);
    const uint32_t rank = cta_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(done + i, 1);
            mbar_init(drained + i, 2 * kGluOutWarps);
        }
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_barrier();
    tc_fence_after();
    let_next_start();
    after_previous();
    const uint32_t tmem = *slot;
    const int64_t step = gridDim.x / 2, first = blockIdx.x / 2;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            // ---- both CTAs: their halves of the operands
            int s = 0;
            uint32_t ph = 1;  // the stages start empty
            for (int64_t id = first; id < a.tiles && ok; id += step) {
                const GluTile t = glu_tile<MODE>(a, id);
                for (int k = t.k0; k < t.k1; ++k) {
                    if (!(ok = mbar_wait(empty + s, ph))) break;
                    unsigned char* sa = smem + s * 2 * kGluOperand;
                    unsigned char* sb = sa + kGluOperand;
                    const int part = k / a.ksteps, kk = (k - part * a.ksteps) * 2 * kGluK;
                    const uint32_t bar = peer_addr(full + s, 0);
                    if (rank == 0) mbar_arrive_expect_tx(full + s, 4 * kGluOperand);
                    auto fetch = [&](unsigned char* to, const CUtensorMap* map, bool kmajor, int row, int kk) {
                        if (a.wide) {
                            tma_pair_3d(to, map, kmajor ? row : kk, (kmajor ? kk : row) / 64, bar);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                tma_pair_2d(to + i * kGluHalf, map, kmajor ? kk + i * 64 : row + i * 64, kmajor ? row : kk, bar);
                        }
                    };
                    const int half = (int)rank * 128;
                    fetch(sa, &maps.a[MODE == kGluFwd ? 0 : MODE == kGluDx ? part : t.problem], AK, (int)t.m + half,
                          MODE == kGluDw ? kk + part * a.lo : kk);
                    fetch(sb, &maps.b[MODE == kGluFwd ? rank : MODE == kGluDx ? part : 0], BK, (int)t.n + (MODE == kGluFwd ? 0 : half), kk);
                    if (++s == ST) s = 0, ph ^= 1;
                }
            }
            // every stage has been released: no arrival is under way to a CTA that has ended
            const int end = s;
            const uint32_t end_ph = ph;
            for (int i = 0; i < ST && ok; ++i) {
                ok = mbar_wait(empty + s, ph);
                if (++s == ST) s = 0, ph ^= 1;
            }
            // a wait that ran out: both CTAs' copies land before the pair ends
            for (int i = 0; i < ST && !ok && rank == 0 && mbar_wait(full + i, i < end ? end_ph ^ 1 : end_ph); ++i) {}
        }
    } else if (warp == 1 && rank == 0) {
        if (lane == 0) {
            // ---- the first CTA: the products of both
            int s = 0;
            uint32_t ph = 0, acc = 0, acc_ph = 1;
            for (int64_t id = first; id < a.tiles && ok; id += step) {
                const GluTile t = glu_tile<MODE>(a, id);
                if (!(ok = mbar_wait(drained + acc, acc_ph))) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * 256;
                for (int k = t.k0; k < t.k1; ++k) {
                    if (!(ok = mbar_wait(full + s, ph))) break;
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + s * 2 * kGluOperand);
                    const uint64_t da = swizzled_desc(sa, AK, kGluHalf), db = swizzled_desc(sa + kGluOperand, BK, kGluHalf);
#pragma unroll
                    for (int j = 0; j < 2 * kGluK / 16; ++j) {
                        // the next 64 k of a K-major operand are a half on
                        const uint32_t split = j / 4 * kGluHalf + j % 4 * 32, ka = AK ? split : j * 2048, kb = BK ? split : j * 2048;
                        mma_bf16<2>(d, da + (ka >> 4), db + (kb >> 4), IDESC, k > t.k0 || j > 0);
                    }
                    mma_commit_pair(empty + s);
                    if (++s == ST) s = 0, ph ^= 1;
                }
                if (!ok) break;
                mma_commit_pair(done + acc);
                if (++acc == 2) acc = 0, acc_ph ^= 1;
            }
        }
    } else if (warp >= 4) {
        // ---- both CTAs: accumulators to memory.  A warp: 32 of this CTA's 128 rows, a thread each, and half of the columns.
        uint32_t acc = 0, ph = 0;
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        unsigned char* st = staging + (warp - 4) * (SAVE ? 2 : 1) * 2048;
        for (int64_t id = first; id < a.tiles; id += step) {
            const GluTile t = glu_tile<MODE>(a, id);
            ok = mbar_wait(done + acc, ph);
            if (!(ok = __all_sync(kFullMask, ok))) break;
            tc_fence_after();
            const uint32_t col = tmem + ((uint32_t)(32 * quarter) << 16) + acc * 256;
            const int64_t row = t.m + (int64_t)rank * 128 + 32 * quarter;  // the warp's first
            const int rows = (int)max((int64_t)0, min((int64_t)32, a.M - row));
            // 64 bytes of the warp's rows, staged, to column c of an output of `esize`-byte elements
            auto out = [&](unsigned char* from, void* to, int64_t c, int esize) {
                glu_rows_out(from, static_cast<unsigned char*>(to) + (row * a.N + c) * esize, a.N * esize, rows,
                             (int)min((int64_t)64, (a.N - c) * esize), lane);
            };
            if constexpr (MODE == kGluFwd) {
                for (int c0 = half * 64; c0 < half * 64 + 64 && t.n + c0 < a.N; c0 += 32) {
                    float g[32], u[32];
                    tmem_ld16(col + c0, *reinterpret_cast<float(*)[16]>(g));
                    tmem_ld16(col + c0 + 16, *reinterpret_cast<float(*)[16]>(g + 16));
                    tmem_ld16(col + 128 + c0, *reinterpret_cast<float(*)[16]>(u));
                    tmem_ld16(col + 128 + c0 + 16, *reinterpret_cast<float(*)[16]>(u + 16));
                    tmem_wait_ld();
                    if constexpr (SAVE) {
                        // the upper halves, then h and the next bytes
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            alignas(16) uint32_t x[4], y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int e = p * 8 + 2 * k;
                                x[k] = __byte_perm(__float_as_uint(g[e]), __float_as_uint(g[e + 1]), 0x7632);
                                y[k] = __byte_perm(__float_as_uint(u[e]), __float_as_uint(u[e + 1]), 0x7632);
                            }
                            *glu_piece(st, lane, p) = *reinterpret_cast<const uint4*>(x);
                            *glu_piece(st + 2048, lane, p) = *reinterpret_cast<const uint4*>(y);
                        }
                        __syncwarp();
                        out(st, a.saved, t.n + c0, 2);
                        out(st + 2048, a.saved + a.M * a.N, t.n + c0, 2);
                        __syncwarp();
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            alignas(16) uint32_t x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int e = p * 8 + 2 * k;  // bytes 1 of g, u, g, u
                                const uint32_t lo = __byte_perm(__float_as_uint(g[e]), __float_as_uint(u[e]), 0x0051);
                                const uint32_t hi = __byte_perm(__float_as_uint(g[e + 1]), __float_as_uint(u[e + 1]), 0x0051);
                                x[k] = __byte_perm(lo, hi, 0x5410);
                            }
                            *glu_piece(st + 2048, lane, p) = *reinterpret_cast<const uint4*>(x);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        alignas(16) uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int e = p * 8 + 2 * k;
                            w[k] = bf16_pair(glu_act<ACT>(g[e]) * u[e], glu_act<ACT>(g[e + 1]) * u[e + 1]);
                        }
                        *glu_piece(st, lane, p) = *reinterpret_cast<const uint4*>(w);
                    }
                    __syncwarp();
                    out(st, a.out[0], t.n + c0, 2);
                    if constexpr (SAVE) out(st + 2048, a.saved + 2 * a.M * a.N, t.n + c0, 2);
                    __syncwarp();
                }
            } else {
                void* to = t.problem ? a.out[1] : a.out[0];
                float* part = a.partial + ((int64_t)t.problem * a.splits + t.split) * a.M * a.N;
                const bool joined = a.partial != nullptr, narrow = !joined && !a.out_f32;
                for (int c0 = half * 128; c0 < half * 128 + 128 && t.n + c0 < a.N; c0 += 32) {
                    float x[2][16];
                    tmem_ld16(col + c0, x[0]);
                    tmem_ld16(col + c0 + 16, x[1]);
                    tmem_wait_ld();
                    if (narrow) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float* y = x[p >> 1] + (p & 1) * 8;
                            *glu_piece(st, lane, p) = make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]),
                                                                 bf16_pair(y[6], y[7]));
                        }
                        __syncwarp();
                        out(st, to, t.n + c0, 2);
                        __syncwarp();
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
#pragma unroll
                            for (int p = 0; p < 4; ++p) *glu_piece(st, lane, p) = reinterpret_cast<const uint4*>(x[i])[p];
                            __syncwarp();
                            if (t.n + c0 + 16 * i < a.N) out(st, joined ? static_cast<void*>(part) : to, t.n + c0 + 16 * i, 4);
                            __syncwarp();
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(peer_addr(drained + acc, 0));
            if (++acc == 2) acc = 0, ph ^= 1;
        }
    }
    if (!ok && lane == 0 && a.status != nullptr) atomicCAS(a.status, GDN_OK, GDN_ERR_TIMEOUT);
    __syncwarp();
    cluster_barrier();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ------------------------------------------------------------- few tokens
constexpr int kGluFewStages = 24;  // most stages

struct GluFewArgs {
    int32_t T, F, ksteps;          // ksteps: of 64 columns
    int32_t rows, stages, chunks;  // units of a block (a multiple of 8, at most 64); stages; 64 columns in each
    void* h;
    uint16_t* saved;
    int32_t* status;
};

struct GluFewMaps {
    CUtensorMap x, wg, wu;
};

// Shared memory of 64 columns: the units of Wg, the same of Wu, NB tokens
__host__ __device__ constexpr uint32_t glu_few_chunk(int NB, int rows) { return (uint32_t)(2 * rows + NB) * 128; }
// The stages; the product reads 128 rows from each one's start on, whose rows behind the weights' count for
// nothing; the results lie where the stages were.
__host__ __device__ inline uint32_t glu_few_tiles(int NB, int rows, int stages, int chunks)
{
    const uint32_t tiles = stages * chunks * glu_few_chunk(NB, rows) + kGluHalf, results = 2 * NB * 64 * 4;
    return tiles > results ? tiles : results;
}

template <int NB, int ACT>
__global__ void __launch_bounds__(kGluThreads, 1) k_glu_few(const __grid_constant__ GluFewMaps maps, const GluFewArgs a)
{
    constexpr uint32_t COLS = NB < 32 ? 32 : NB;
    constexpr uint32_t IDESC = bf16_idesc(128, NB, true, true);
    extern __shared__ unsigned char glu_smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(glu_smem_raw) + 1023) & ~(uintptr_t)1023);
    const int ST = a.stages, C = a.chunks;
    const uint32_t chunk = glu_few_chunk(NB, a.rows);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + glu_few_tiles(NB, a.rows, ST, C));
    uint64_t* empty = full + kGluFewStages;
    uint64_t* done = empty + kGluFewStages;
    uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t S;  // blocks that share the K axis
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
    const uint32_t rank = cta_rank();
    const int f0 = blockIdx.x / S * a.rows, t0 = blockIdx.y * NB;
    const int all = (a.ksteps + C - 1) / C, first = (int)((int64_t)all * rank / S);
    const int turns = (int)((int64_t)all * (rank + 1) / S) - first;  // at least one: the host sees to it
    if (lane == 0 && (warp == 0 || warp == 2 || warp == 3))
        prefetch_map(warp == 0 ? &maps.wg : warp == 2 ? &maps.wu : &maps.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        mbar_init(done, 1);
    }
    if (warp == 2) tmem_alloc(slot, COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    let_next_start();
    after_previous();
    const uint32_t tmem = *slot;
    bool ok = true;
    if (warp == 0 || warp == 2 || warp == 3) {
        if (lane == 0) {
            // one warp for each operand; the first announces the bytes of all
            const CUtensorMap* map = warp == 0 ? &maps.wg : warp == 2 ? &maps.wu : &maps.x;
            const uint32_t at = warp == 0 ? 0 : warp == 2 ? a.rows * 128 : 2 * a.rows * 128;
            const int y = warp == 3 ? t0 : f0;
            int s = 0;
            uint32_t ph = 1;
            for (int k = 0; k < turns; ++k) {
                if (!(ok = mbar_wait(empty + s, ph))) break;
                if (warp == 0) mbar_arrive_expect_tx(full + s, C * chunk);
                for (int c = 0; c < C; ++c)
                    tma_2d(smem + (s * C + c) * chunk + at, map, ((first + k) * C + c) * kGluK, y, full + s);
                if (++s == ST) s = 0, ph ^= 1;
            }
            // a wait that ran out: the copies land before the block ends
            for (int i = 0; i < ST && !ok && mbar_wait(full + i, i < s ? ph ^ 1 : ph); ++i) {}
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int k = 0; k < turns; ++k) {
                if (!(ok = mbar_wait(full + s, ph))) break;
                tc_fence_after();
                for (int c = 0; c < C; ++c) {
                    const uint32_t p = smem_addr(smem + (s * C + c) * chunk);
                    const uint64_t dw = swizzled_desc(p, true), dx = swizzled_desc(p + 2 * a.rows * 128, true);
#pragma unroll
                    for (int j = 0; j < kGluK / 16; ++j) mma_bf16<1>(tmem, dw + 2 * j, dx + 2 * j, IDESC, k > 0 || c > 0 || j > 0);
                }
                mma_commit(empty + s);
                if (++s == ST) s = 0, ph ^= 1;
            }
            mma_commit(done);
        }
    }
    __syncwarp();
    if (!mbar_wait(done, 0)) ok = false;
    tc_fence_after();
    ok = __syncthreads_and(ok);
    // accumulators to shared memory: [2][tokens][64 units], half of the tokens by either four warps
    float* out = reinterpret_cast<float*>(smem);
    {
        const int r = 32 * (warp & 3) + lane;
        const uint32_t col = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int up = r >= a.rows;  // rows behind both are written nowhere
        float* to = out + up * NB * 64 + (r - up * a.rows);
        for (int c = (warp >> 2) * 16; c < NB && t0 + c < a.T; c += 32) {
            float x[16];
            tmem_ld16(col + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (r < 2 * a.rows) to[(c + j) * 64] = x[j];
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, COLS);
    if (S > 1) {
        // a wait that ran out counts for the whole cluster
        if (threadIdx.x == 0) *slot = ok;
        cluster_barrier();
        for (uint32_t q = 0; q < S; ++q) {
            uint32_t good;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(good) : "r"(peer_addr(slot, q)) : "memory");
            ok = ok && good;
        }
    }
    if (!ok && threadIdx.x == 0 && a.status != nullptr) atomicCAS(a.status, GDN_OK, GDN_ERR_TIMEOUT);
    const int r = threadIdx.x & 63, f = f0 + r;
    const int64_t plane = (int64_t)a.T * a.F;
    if (ok && r < a.rows && f < a.F) {  // else the outputs are left as they are
        auto finish = [&](int t, float g, float u) {
            const int64_t at = (int64_t)(t0 + t) * a.F + f;
            if (a.saved != nullptr) glu_pack(g, u, a.saved[at], a.saved[plane + at], a.saved[2 * plane + at]);
            static_cast<__nv_bfloat16*>(a.h)[at] = __float2bfloat16_rn(glu_act<ACT>(g) * u);
        };
        const int last = min(NB, a.T - t0), group = threadIdx.x >> 6;
        if (S == 1) {
#pragma unroll 4
            for (int t = group; t < last; t += kGluThreads / 64) finish(t, out[t * 64 + r], out[(NB + t) * 64 + r]);
        } else {
            // tokens round the cluster
            for (int t = (int)rank + (int)S * group; t < last; t += (int)S * (kGluThreads / 64)) {
                float g = 0.0f, u = 0.0f;
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q) {
                    if (q < S) {
                        const uint32_t p = peer_addr(out + t * 64 + r, q);
                        float x, y;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(p) : "memory");
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(p + NB * 64 * 4) : "memory");
                        g += x;
                        u += y;
                    }
                }
                finish(t, g, u);
            }
        }
    }
    if (S > 1) {
        __syncwarp();
        cluster_barrier();  // no block ends while another reads it
    }
}

// ------------------------------------------------------------- elementwise parts
// Eight 2-byte elements at p, of the tensor [base, end): two aligned accesses where they lie within it
__device__ __forceinline__ uint4 glu_load8(const uint16_t* p, const uint16_t* base, const uint16_t* end, int64_t count)
{
    const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint16_t* q = p - s / 2;
    if (s == 0 && count >= 8) return *reinterpret_cast<const uint4*>(p);
    if (q >= base && q + 16 <= end) {
        const uint4* v = reinterpret_cast<const uint4*>(q);
        return s == 0 ? v[0] : bytes_at(v[0], v[1], s);
    }
    Vec<uint16_t, 8> v;
#pragma unroll
    for (int k = 0; k < 8; ++k) v.v[k] = k < count ? p[k] : (uint16_t)0;
    return *reinterpret_cast<const uint4*>(&v);
}

// dg and du, rows ld (a multiple of 8) apart, from dh and what the forward saved; columns from F on are read by nobody.
// LO: what their rounding to bf16 leaves goes into T more rows behind.
// WHOLE: every row of dh and of the planes is whole 16-byte vectors (121 us at 8192 x 8192, the copy rate; else 131).
template <bool WHOLE, int ACT, bool LO>
__global__ void __launch_bounds__(256) k_glu_grad(const uint16_t* __restrict__ dh, int64_t lddh,
                                                  const uint16_t* __restrict__ saved, int64_t T, int64_t F,
                                                  __nv_bfloat16* __restrict__ dg, __nv_bfloat16* __restrict__ du, int64_t ld)
{
    let_next_start();
    after_previous();
    const int64_t per = ld / 8, n = T * per, plane = T * F;
    const uint16_t *dend = dh + (T - 1) * lddh + F, *send = saved + 3 * plane;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per, c = (i - t * per) * 8, left = F - c;
        const uint16_t* s = saved + t * F + c;
        auto load = [&](const uint16_t* p, const uint16_t* base, const uint16_t* end) {
            return WHOLE ? *reinterpret_cast<const uint4*>(p) : glu_load8(p, base, end, left);
        };
        const uint4 d4 = load(dh + t * lddh + c, dh, dend), g4 = load(s, saved, send), u4 = load(s + plane, saved, send),
                    l4 = load(s + 2 * plane, saved, send);
        const __nv_bfloat16* d = reinterpret_cast<const __nv_bfloat16*>(&d4);
        const uint16_t *gh = reinterpret_cast<const uint16_t*>(&g4), *uh = reinterpret_cast<const uint16_t*>(&u4),
                       *low = reinterpret_cast<const uint16_t*>(&l4);
        float x[8], y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float g, u, f, slope;
            glu_unpack(gh[k], uh[k], low[k], g, u);
            glu_act2<ACT>(g, f, slope);
            const float e = to_f<__nv_bfloat16>(d[k]);
            x[k] = e * u * slope;
            y[k] = e * f;
        }
        store_vec<__nv_bfloat16, 8>(dg + t * ld + c, x);
        store_vec<__nv_bfloat16, 8>(du + t * ld + c, y);
        if constexpr (LO) {
            auto left_over = [](float v) {
                const float r = to_f<__nv_bfloat16>(__float2bfloat16_rn(v));
                return isfinite(r) ? v - r : 0.0f;
            };
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = left_over(x[k]), y[k] = left_over(y[k]);
            store_vec<__nv_bfloat16, 8>(dg + (T + t) * ld + c, x);
            store_vec<__nv_bfloat16, 8>(du + (T + t) * ld + c, y);
        }
    }
}

// Matrices whose rows are not whole 16 bytes, into rows that are (ldd: a multiple of 8); one by blockIdx.y.
struct GluAlign {
    const uint16_t* src[3];
    uint16_t* dst[3];
    int64_t lds[3], rows[3];
    int64_t cols, ldd;
};
__global__ void __launch_bounds__(256) k_glu_align(const GluAlign a)
{
    let_next_start();
    const int m = blockIdx.y;
    const uint16_t* src = m == 0 ? a.src[0] : m == 1 ? a.src[1] : a.src[2];
    uint16_t* dst = m == 0 ? a.dst[0] : m == 1 ? a.dst[1] : a.dst[2];
    const int64_t lds = m == 0 ? a.lds[0] : m == 1 ? a.lds[1] : a.lds[2], rows = m == 0 ? a.rows[0] : m == 1 ? a.rows[1] : a.rows[2];
    const int64_t per = a.ldd / 8, n = rows * per;
    const uint16_t* end = src + (rows - 1) * lds + a.cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        *reinterpret_cast<uint4*>(dst + r * a.ldd + c) = glu_load8(src + r * lds + c, src, end, a.cols - c);
    }
}

// The sums of the splits' partial products, in ascending order.
template <typename OT>
__global__ void __launch_bounds__(256) k_glu_join(const float* __restrict__ part, int splits, int64_t n, OT* __restrict__ out0,
                                                  OT* __restrict__ out1, int problems)
{
    let_next_start();
    after_previous();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * problems; i += (int64_t)gridDim.x * 256) {
        const int64_t p = i / n, e = i - p * n;
        const float* s = part + p * splits * n + e;
        float x = 0.0f;
        for (int k = 0; k < splits; ++k) x += s[k * n];
        (p ? out1 : out0)[e] = from_f<OT>(x);
    }
}

}  // namespace gdn

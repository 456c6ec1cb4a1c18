// k_policy.cuh -- the clipped policy loss with a KL term on rows of logits: log-probabilities, losses and
// the logits' gradient (sm_100a).
//
//     lp = z_y / tau - log sum_v e^(z_v / tau),  ratio = e^(lp - old)
//     loss = -min(ratio A, clip(ratio, 1 - lo, 1 + hi) A) + kl (e^(ref - lp) - (ref - lp) - 1)
//     dz_v = dloss d (1[v = y] - e^(z_v / tau) / sum) / tau,  d = dloss/dlp
//
// One block walks a row twice: running maximum and sum, then the gradient.  A warp of its own streams the row's tiles
// into a ring in shared memory with bulk copies; the tiles of a row's end are still there when the second walk
// begins with them, and only what the ring does not hold is fetched again (from L2).  The copies run
// ahead over the end of the walks and of the rows, so that memory does not wait for the two block-wide sums per row.
// Bound by the bytes (the logits once, with their gradient twice) next to 2^x: one per logit, with the gradient two, which
// alone would take 235 us of the 395 to 400 us for 4096 x 131072 bf16 (5.4 TB/s; the special-function unit at 16 per cycle
// and SM).  777 x 50021 fp32, losses alone: 34 us (4.6 TB/s).  Log-probabilities of 64 x 131072 bf16 take 10 us, of one
// row 8: latency.
// (Many rows cut over clusters of up to 8 blocks, wholly in shared memory, waited for each other: 495 us at
// 4096 x 131072 bf16, whether with the cluster's barrier or with exchanges a row ahead.)
//
// Where there are few rows, a cluster of blocks shares each (64 x 131072: 4): a block walks its part of the tiles, then all
// read the others' maxima and sums in distributed shared memory.
//
// The partition of a row, up to 8 parts, follows from the vocabulary and the type alone: a thread's elements are the same
// whatever the row's address and stride, and their parts' sums are joined one after the other, whether they lie in one
// block or in several.  So a row's log-probability has the same bits in every
// batch, in a strided view or a dense tensor, in the forward and with the gradient.  A ratio between
// a rollout and a trainer that saw the same logits is then exactly 1.
#pragma once

#include "cluster.cuh"
#include "layer_common.cuh"
#include "tma.cuh"

namespace gdn {

constexpr int kPolicyVecs = 4;    // 16-byte vectors of a tile per thread

struct PolicyArgs {
    const void* z;
    int64_t ldz;
    const int64_t* y;
    const float *old, *ref, *adv, *dloss;  // old == null: log-probabilities only
    float lo, hi, kl;                      // borders of the ratio, weight of the KL term
    float c, inv_tau;                      // log2(e) / tau, 1 / tau
    int64_t T;
    int32_t V;
    float *loss, *lp;
    void* dz;
    int32_t* status;
};

// n bytes, a multiple of 16, both addresses 16-byte aligned
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* mbar, uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                     smem_addr(dst)), "l"(src), "r"(n), "r"(smem_addr(mbar)), "l"(policy)
                 : "memory");
}

// The running maximum m is in units of log2, max(z) c with c = log2(e) / tau, and a row's exponents are fma(z, c, -m): they share the
// rounding of m, at most 32 where |m| is below 2^30, which the sum takes out again.  Beyond, it would leave the range of 2^x.
// Maxima start at -2^30, below which nothing is told apart, and a row whose maximum ends there or at 2^30 and above (one that a mask
// of -1e10 or of the type's lowest value fills) is walked once more (policy_far).
constexpr float kPolicyFar = 1073741824.0f;

// The largest of a thread's packed values.
template <typename T, int E>
struct PolicyMax;
template <>
struct PolicyMax<__nv_bfloat16, 8> {
    __nv_bfloat162 m = __float2bfloat162_rn(-INFINITY);
    __device__ __forceinline__ void add(const Vec<__nv_bfloat16, 8>& v)
    {
        const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
        m = __hmax2(m, __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    }
    __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct PolicyMax<float, 4> {
    float m = -INFINITY;
    __device__ __forceinline__ void add(const Vec<float, 4>& v)
    {
        m = fmaxf(m, fmaxf(fmaxf(v.v[0], v.v[1]), fmaxf(v.v[2], v.v[3])));
    }
    __device__ __forceinline__ float get() const { return m; }
};

// The maximum and the sum of 2^(x - maximum) over N neighbouring lanes, from each one's own; the same in all of them.
template <int N>
__device__ __forceinline__ void policy_join(float& m, float& sum)
{
    float M = m;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
    sum *= ex2(m - M);
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    m = M;
}

// E elements that are written once and not read here: first to leave L2
template <typename T, int E>
__device__ __forceinline__ void store_once(T* p, const f2x (&x)[E / 2])
{
    Vec<T, E> r;
    pstore<T, E>(r.v, x);
    const uint4 u = *reinterpret_cast<const uint4*>(&r);
    asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
}

__host__ __device__ constexpr int policy_tile_bytes(int NT) { return NT * kPolicyVecs * 16; }
// a tile that starts s bytes into its first 16, and as many behind its last
__host__ __device__ constexpr int policy_slot_bytes(int NT) { return policy_tile_bytes(NT) + 32; }

// Tiles in the ring with so many blocks per SM; all but two of them stay for the second walk.
__host__ __device__ constexpr int policy_slots(int resident) { return resident == 2 ? 6 : 4; }

// Parts of a row of n tiles: a power of two (its logarithm), of at least 4 tiles each, or 2 where there are two parts.  (Parts of
// 2 tiles throughout: 64 x 131072 bf16 10.9 us in place of 9.9, 1 x 131072 7.6 and 7.8; 32 x 50021, 7 tiles, 7.6 and 9.1.)
constexpr int kPolicyParts = 8;
__host__ __device__ constexpr int policy_parts_log(int n) { return n >= 32 ? 3 : n >= 16 ? 2 : n >= 4 ? 1 : 0; }

// The maximum and sum of what lies behind, joined to those of what lies before
__device__ __forceinline__ void policy_add(float& m, float& sum, float m1, float sum1)
{
    const float M = fmaxf(m, m1);
    sum = __fmaf_rn(sum1, ex2(m1 - M), sum * ex2(m - M));
    m = M;
}

// A row whose maximum is far off, by NT threads: the maximum M itself and how many logits equal it, which are all that count: logits that
// differ there differ by 64 or more in units of log2.  n: as a sum relative to M, not a number where a logit is not or M is infinite.
// (As a call of its own it cost every row: losses of 200000 x 1000 301 us in place of 293.)
template <typename T, int NT>
__device__ __forceinline__ float2 policy_far(const T* z, int V, float* wm, float* ws)
{
    const int tid = threadIdx.x, lane = tid & 31;
    auto together = [] { asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory"); };
    float M = -INFINITY, bad = 0.0f;
#pragma unroll 1
    for (int i = tid; i < V; i += NT) {
        const float x = to_f<T>(z[i]);
        M = fmaxf(M, x);
        if (x != x) bad = x;
    }
    auto warps = [&](float x, float* w, auto join) {  // over all threads, the same in each
        for (int o = 16; o > 0; o >>= 1) x = join(x, __shfl_xor_sync(kFullMask, x, o));
        together();
        if (lane == 0) w[tid >> 5] = x;
        together();
        x = w[0];
        for (int i = 1; i < NT / 32; ++i) x = join(x, w[i]);
        return x;
    };
    M = warps(M, wm, [](float x, float y) { return fmaxf(x, y); });
    int count = 0;
#pragma unroll 1
    for (int i = tid; i < V; i += NT) count += to_f<T>(z[i]) == M;
    // (the counts are whole: in two halves of 16 bits exact in fp32, whatever the order)
    float n = warps((float)(count >> 16) * 65536.0f, ws, [](float x, float y) { return x + y; }) +
        warps((float)(count & 0xffff), wm, [](float x, float y) { return x + y; });
    n += warps(bad, ws, [](float x, float y) { return x + y; });
    return make_float2(M, isinf(M) ? M - M : n);
}

// e^g - 1 - g without the cancellation, and its derivative for -g.  Within 1/2: g^2 (1/2! + g/3! + .. + g^7/9!), what is left out is
// below 2^-29 of it; beyond, the difference is at least a quarter of e^g - 1.
__device__ __forceinline__ float policy_kl(float g, float& slope)
{
    if (__builtin_expect(!(fabsf(g) <= 0.5f), 0)) {
        const float e1 = expm1f(g);
        slope = -e1;
        return e1 - g;
    }
    const float g2 = g * g;  // in pairs: a row waits for it
    float p = __fmaf_rn(1.0f / 362880.0f, g, 1.0f / 40320.0f);
    p = __fmaf_rn(p, g2, __fmaf_rn(1.0f / 5040.0f, g, 1.0f / 720.0f));
    p = __fmaf_rn(p, g2, __fmaf_rn(1.0f / 120.0f, g, 1.0f / 24.0f));
    p = __fmaf_rn(p, g2, __fmaf_rn(1.0f / 6.0f, g, 0.5f));
    p *= g2;
    slope = -(g + p);
    return p;
}

// NT threads walk, 32 more fetch; `RES` blocks per SM.  ALIGNED: every row of the logits and of the gradient is whole
// 16-byte vectors.  SPLIT: a cluster of blocks per row, each with the same number of the row's parts.
template <typename T, bool BWD, bool ALIGNED, int NT, int RES, bool SPLIT>
__global__ void __launch_bounds__(NT + 32, RES) k_policy(const PolicyArgs a)
{
    constexpr int E = 16 / (int)sizeof(T);  // elements of a vector
    constexpr int NV = kPolicyVecs, K = policy_slots(RES), TILE = NT * NV * E, SLOT = policy_slot_bytes(NT), WARPS = NT / 32;
    constexpr long long LIMIT = 1ll << 31;
    extern __shared__ __align__(128) unsigned char policy_smem[];  // tiles, each at its global address mod 16
    __shared__ __align__(8) uint64_t full[K], empty[K], joined;
    __shared__ float wm[WARPS], ws[WARPS], target_logit;
    __shared__ volatile int lost;           // a wait that ran out: nothing is written from then on
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tiles = (int)(((unsigned)a.V + TILE - 1) / TILE), lg = NT == 256 ? policy_parts_log(tiles) : 0, parts = 1 << lg;  // of a row
    int S = 1, rank = 0;  // blocks of a row, and which of them this is
    if constexpr (SPLIT) {
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
        rank = (int)cta_rank();
    }
    const int mine = parts / S, part0 = mine * rank;  // this block's parts, and its tiles
    const int first = SPLIT ? tiles * part0 >> lg : 0, last = SPLIT ? tiles * (part0 + mine) >> lg : tiles, n = last - first;
    const int64_t row0 = SPLIT ? blockIdx.x / S : blockIdx.x, rows = SPLIT ? a.T : gridDim.x;  // the block's first row and its step
    const int stay = BWD ? min(n, K - 2) : 0, again = BWD ? n - stay : 0;
    float2* found = reinterpret_cast<float2*>(policy_smem + K * SLOT);  // SPLIT: [mine][NT] maxima and sums, for the cluster
    if (tid == 0) {
        for (int i = 0; i < K; ++i) {
            mbar_init_cta(full + i, 1);
            mbar_init_cta(empty + i, WARPS);
        }
        if constexpr (SPLIT) mbar_init_cta(&joined, S);
        lost = 0;
    }
    if constexpr (SPLIT) cluster_barrier();
    else __syncthreads();
    let_next_start();
    after_previous();
    auto target = [&](int64_t row) -> int {  // -1: a row that takes no part
        if (row >= a.T) return -1;
        const int64_t y = a.y[row];
        return y >= a.V || y < 0 ? -1 : (int)y;
    };
    auto misplaced = [&](int64_t row) -> int {
        return ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(static_cast<const T*>(a.z) + row * a.ldz) & 15);
    };
    int slot = 0;
    uint32_t phase = 0;

    if (warp == WARPS) {
        // ---- the copies: a row's tiles in order, then those that did not stay
        phase = 1;  // the slots start empty
        // what is fetched again stays in L2 until then, before what is read or written once
        uint64_t keep, once;
        asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        int y_next = target(row0);
        for (int64_t row = row0; row < a.T; row += rows) {
            const int y = y_next;
            y_next = target(row + rows);
            if (a.status != nullptr && lane == 0 && a.y[row] >= a.V) atomicCAS(a.status, GDN_OK, GDN_ERR_DEVICE_INPUT);
            if (y < 0) continue;
            const T* z = static_cast<const T*>(a.z) + row * a.ldz;
            const int s = misplaced(row);
            for (int t = 0; t < n + again; ++t) {
                const int tile = first + (t < n ? t : t - n);
                const int len = min(TILE, a.V - tile * TILE);
                const T* src = z + (int64_t)tile * TILE;
                unsigned char* dst = policy_smem + slot * SLOT;
                if (lost || !mbar_wait_bounded(empty + slot, phase, LIMIT)) {
                    lost = 1;
                    break;
                }
                // Whole 16-byte granules, those that the tile shares with its neighbours too; what shares one with
                // the bytes before or behind the row comes element by element.
                int from = -s, to = len * (int)sizeof(T);  // bytes
                if constexpr (!ALIGNED) {
                    T* at = reinterpret_cast<T*>(dst + s);
                    if (s != 0 && tile == 0) {
                        from = min(16 - s, to);
                        if (lane * (int)sizeof(T) < from) at[lane] = src[lane];
                    }
                    int end = ((s + to + 15) & ~15) - s;
                    const int rest = a.V - tile * TILE;  // to the row's end
                    if (end > rest * (int)sizeof(T)) {
                        end = max(from, ((s + to) & ~15) - s);
                        const int i = max(end, 0) / (int)sizeof(T) + lane;
                        if (lane < E && i < rest) at[i] = src[i];
                    }
                    if (len + lane < (len + E - 1) / E * E) at[len + lane] = from_f<T>(-INFINITY);  // fills the row's last vector
                    to = end;
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(full + slot, (uint32_t)(to - from));
                    if (to > from)
                        bulk_load(dst + s + from, reinterpret_cast<const unsigned char*>(src) + from, (uint32_t)(to - from), full + slot, t < again ? keep : once);
                }
                if (++slot == K) slot = 0, phase ^= 1;
            }
            if (lost) break;
        }
        // every copy has landed before the block ends, whether the walks wait for it or have given up
        for (int i = 0; i < K && mbar_wait_bounded(full + i, i < slot ? phase ^ 1 : phase, LIMIT); ++i) {}
        if constexpr (SPLIT) {
            __syncwarp();
            cluster_barrier();
        }
        return;
    }

    // ---- the walks
    const f2x c2 = pk2(a.c, a.c);
    auto wait = [&] {
        if (!lost && !mbar_wait_bounded(full + slot, phase, LIMIT)) lost = 1;
    };
    auto release = [&](int at) {
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(empty + at)) : "memory");
    };
    auto advance = [&] {
        if (++slot == K) slot = 0, phase ^= 1;
    };
    auto together = [] { asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory"); };  // the walking threads
    int y_next = target(row0);
    for (int64_t row = row0; row < a.T; row += rows) {
        const int y = y_next;
        y_next = target(row + rows);
        T* out = static_cast<T*>(a.dz) + row * a.V;
        if (y < 0) {  // nothing is read
            if (tid == 0 && rank == 0) {
                if (a.loss != nullptr) a.loss[row] = 0.0f;
                if (a.lp != nullptr) a.lp[row] = 0.0f;
            }
            if constexpr (BWD) {
                const int64_t begin = (int64_t)first * TILE, end = min((int64_t)last * TILE, (int64_t)a.V);
                if constexpr (ALIGNED) {
                    for (int64_t i = begin / E + tid; i < end / E; i += NT) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
                } else {
                    for (int64_t i = begin + tid; i < end; i += NT) out[i] = from_f<T>(0.0f);
                }
            }
            continue;
        }
        // what the row's end needs, on its way from here on
        const float old = a.old != nullptr ? a.old[row] : 0.0f, adv = a.old != nullptr ? a.adv[row] : 0.0f;
        const float ref = a.ref != nullptr ? a.ref[row] : 0.0f, dloss = BWD ? a.dloss[row] : 0.0f;
        const int s = misplaced(row);
        // (the tile that holds it may be another block's, which may put the gradient in its place)
        [[maybe_unused]] const float split_target = SPLIT ? to_f<T>((static_cast<const T*>(a.z) + row * a.ldz)[y]) : 0.0f;
        auto vec = [&](int i) {
            const uint4* p = reinterpret_cast<const uint4*>(policy_smem + slot * SLOT) + i;
            uint4 r = p[0];
            if (!ALIGNED && s != 0) r = bytes_at(r, p[1], s);
            return *reinterpret_cast<const Vec<T, E>*>(&r);
        };
        // ---- the first walk: running maximum (in units of log2) and sum
        float m = -kPolicyFar, sum = 0.0f, before = -kPolicyFar, before_sum = 0.0f;
        const int slot0 = slot;
        const uint32_t phase0 = phase;
        int part = part0, part_end = tiles * (part + 1) >> lg;
        for (int t = first; t < last; ++t) {
            if (t == part_end) {
                if constexpr (SPLIT) found[(part - part0) * NT + tid] = make_float2(m, sum);
                else policy_add(before, before_sum, m, sum);
                m = -kPolicyFar, sum = 0.0f;
                part_end = tiles * (++part + 1) >> lg;
            }
            wait();
            auto add = [&](auto whole, int nvec) {
                constexpr bool WHOLE = decltype(whole)::value;
                Vec<T, E> v[NV];
                PolicyMax<T, E> top;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (WHOLE || tid + j * NT < nvec) {
                        v[j] = vec(tid + j * NT);
                        top.add(v[j]);
                    }
                const float M = fmaxf(m, top.get() * a.c);
                sum *= ex2(m - M);
                m = M;
                const f2x b2 = pk2(-M, -M);
                f2x s0 = pk2(0.0f, 0.0f), s1 = s0;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (WHOLE || tid + j * NT < nvec) {
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) {
                            float x0, x1;
                            up2(pfma(pbits<T, E>(v[j], k), c2, b2), x0, x1);
                            f2x& to = k & 1 ? s1 : s0;
                            to = padd(to, pk2(ex2(x0), ex2(x1)));
                        }
                    }
                sum += psum(padd(s0, s1));
            };
            const int len = a.V - t * TILE;
            if (!SPLIT && tid == 0 && y - t * TILE >= 0 && y - t * TILE < TILE)
                target_logit = to_f<T>(reinterpret_cast<const T*>(policy_smem + slot * SLOT + s)[y - t * TILE]);
            if (len >= TILE) add(std::true_type{}, 0);
            else add(std::false_type{}, (len + E - 1) / E);
            if (t - first < n - stay) release(slot);
            advance();
        }
        if constexpr (SPLIT) {
            found[(part - part0) * NT + tid] = make_float2(m, sum);
            together();
            if (tid < S && !lost) mbar_arrive_peer(peer_addr(&joined, tid));
            if (!mbar_wait_cluster(&joined, 0, LIMIT)) lost = 1;  // (one row per cluster)
            for (int p = 0; p < parts; ++p) {
                float m1, sum1;
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(m1), "=f"(sum1)
                             : "r"(peer_addr(found + p % mine * NT + tid, p / mine)) : "memory");
                policy_add(before, before_sum, m1, sum1);
            }
        } else {
            policy_add(before, before_sum, m, sum);
        }
        m = before, sum = before_sum;
        policy_join<32>(m, sum);
        if (lane == 0) wm[warp] = m, ws[warp] = sum;
        together();
        // every warp joins the warps itself
        m = lane < WARPS ? wm[lane] : -kPolicyFar;
        sum = lane < WARPS ? ws[lane] : 0.0f;
        policy_join<32>(m, sum);
        float C = a.c, bm = m;  // exponents are fma(z, C, -bm)
        const float zt = SPLIT ? split_target : target_logit, at = __fmaf_rn(zt, a.c, -m);
        float head = at * 0.69314718055994530942f;  // lp = head - log(sum); where `near`, from log2(sum) with one product
        const bool near = fabsf(m) < kPolicyFar && fabsf(at) < INFINITY;
        if (__any_sync(kFullMask, !near)) {  // (the same for all; a vote costs a row less than a branch that could part its threads)
            if (fabsf(m) < kPolicyFar) {  // a target far below: out of range times log2(e), perhaps not by itself
                head = zt * a.inv_tau - m * 0.69314718055994530942f;
            } else {
                const float2 far = policy_far<T, NT>(static_cast<const T*>(a.z) + row * a.ldz, a.V, wm, ws);
                m = far.x, sum = far.y;
                // the power of two that puts m C, exact, into 2^40..2^41: equal logits differ by 0, others by 2^16 or more
                C = __uint_as_float((294u - (__float_as_uint(m) >> 23 & 0xffu)) << 23);
                bm = m * C;
                // (by halves: the difference may be out of range where its quotient is not)
                head = zt == m ? 0.0f : (0.5f * zt - 0.5f * m) * a.inv_tau * 2.0f;
                if constexpr (SPLIT && BWD) {  // the gradient may take the place of what another block still walks
                    together();
                    if (tid < S && !lost) mbar_arrive_peer(peer_addr(&joined, tid));
                    if (!mbar_wait_cluster(&joined, 1, LIMIT)) lost = 1;
                }
            }
        }
        together();  // the warps' sums have been read
        [[maybe_unused]] float d = 0.0f;
        // without a gradient the other warps go on to the next row (losses of 16384 x 8000 86 us in place of 94)
        if (BWD || warp == 0) {
            const float log_sum = log2f(sum);
            const float lp = near ? (at - log_sum) * 0.69314718055994530942f : head - log_sum * 0.69314718055994530942f;
            float loss = 0.0f;
            if (a.old != nullptr) {
                const float ratio = ex2((lp - old) * kLog2e);
                if (adv != 0.0f) {  // a zero takes no part, whatever the ratio
                    const float free = -adv * ratio, held = -adv * fminf(fmaxf(ratio, a.lo), a.hi);
                    loss = free < held ? held : free;  // not a number where the ratio is not
                    d = free < held ? 0.0f : free;
                }
                if (a.ref != nullptr && a.kl != 0.0f) {  // (0 times a term that overflowed is not a number)
                    float slope;
                    loss = __fmaf_rn(a.kl, policy_kl(ref - lp, slope), loss);
                    d = __fmaf_rn(a.kl, slope, d);
                }
            }
            if (tid == 0 && rank == 0 && !lost) {
                if (a.loss != nullptr) a.loss[row] = loss;
                if (a.lp != nullptr) a.lp[row] = lp;
            }
        }
        if constexpr (BWD) {
            // ---- the second walk: first the tiles that have stayed, then the others
            d *= dloss * a.inv_tau;
            const float scale = -d * rcp(sum);
            const f2x c2 = pk2(C, C), b2 = pk2(-bm, -bm), scale2 = pk2(scale, scale);
            const int so = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(out) & 15);
            const int end_slot = slot;
            const uint32_t end_phase = phase;
            slot = slot0, phase = phase0;
            for (int i = 0; i < n - stay; ++i) advance();
            for (int t = 0; t < n; ++t) {
                const int tile = t < stay ? last - stay + t : first + t - stay;
                if (t == stay) slot = end_slot, phase = end_phase;
                if (t >= stay) wait();
                T* dst = out + (int64_t)tile * TILE;
                const int rest = a.V - tile * TILE, len = min(TILE, rest), yl = y - tile * TILE;  // rest: to the row's end
                const int here = lost ? 0 : (len + E - 1) / E;
                auto gradient = [&](const Vec<T, E>& v, int first, f2x (&o)[E / 2]) {  // of the elements from `first` on
#pragma unroll
                    for (int k = 0; k < E / 2; ++k) {
                        float x0, x1;
                        up2(pfma(pbits<T, E>(v, k), c2, b2), x0, x1);
                        o[k] = pmul(pk2(ex2(x0), ex2(x1)), scale2);
                    }
                    if ((unsigned)(yl - first) < (unsigned)E) {
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) {
                            const int q = yl - first - 2 * k;
                            o[k] = padd(o[k], pk2(q == 0 ? d : 0.0f, q == 1 ? d : 0.0f));
                        }
                    }
                };
                if (ALIGNED || so == s) {
                    // The gradient's 16-byte granules are the logits': the tile's are those that start in it; of the row's
                    // first and last the elements that belong to the row.
                    const int skip = s ? E - s / (int)sizeof(T) : 0;  // elements before the first of them
                    auto granules = [&](auto whole) {
                        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
                        for (int j = 0; j < NV; ++j) {
                            const int i = tid + j * NT, e = skip + i * E;
                            if (WHOLE || e + E <= rest) {
                                const uint4 r = reinterpret_cast<const uint4*>(policy_smem + slot * SLOT)[i + (s != 0)];
                                f2x o[E / 2];
                                gradient(*reinterpret_cast<const Vec<T, E>*>(&r), e, o);
                                store_once<T, E>(dst + e, o);
                            }
                        }
                    };
                    if (here > 0) {
                        if (rest >= TILE + skip) granules(std::true_type{});
                        else granules(std::false_type{});
                        if (!ALIGNED) {
                            const int last = rest >= TILE + skip ? 0 : max(0, (rest - skip) / E);  // granules of the row's end
                            const int e = tid < E ? (tile == 0 && tid < min(skip, rest) ? tid : -1)
                                                  : tid < 2 * E && rest < TILE + skip && skip + last * E + tid - E < rest ? skip + last * E + tid - E : -1;
                            if (e >= 0) {
                                const float x = to_f<T>(reinterpret_cast<const T*>(policy_smem + slot * SLOT + s)[e]);
                                const float g = ex2(__fmaf_rn(x, C, -bm)) * scale;
                                dst[e] = from_f<T>(e == yl ? g + d : g);  // as in `gradient`: the same bits at every address
                            }
                        }
                    }
                } else {
                    for (int j = 0; j < NV; ++j) {
                        const int i = tid + j * NT;
                        if (i < here) {
                            f2x o[E / 2];
                            gradient(vec(i), i * E, o);
                            Vec<T, E> r;
                            pstore<T, E>(r.v, o);
#pragma unroll
                            for (int k = 0; k < E; ++k)
                                if (i * E + k < len) dst[i * E + k] = r.v[k];
                        }
                    }
                }
                release(slot);
                advance();
            }
            if (again == 0) slot = end_slot, phase = end_phase;
        }
    }
    if (lost && tid == 0 && a.status != nullptr) atomicCAS(a.status, GDN_OK, GDN_ERR_TIMEOUT);
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_barrier();  // no block ends while another reads it
    }
}

}  // namespace gdn

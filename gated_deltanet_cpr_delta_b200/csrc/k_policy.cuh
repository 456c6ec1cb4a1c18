// k_policy.cuh -- the clipped policy loss with a KL term on rows of logits: log-probabilities, losses and
// the logits' gradient (sm_100a).
//
//     lp = z_y / tau - log sum_v e^(z_v / tau),  ratio = e^(lp - old)
//     loss = -min(ratio A, clip(ratio, 1 - lo, 1 + hi) A) + kl (e^(ref - lp) - (ref - lp) - 1)
//     dz_v = dloss d (1[v = y] - e^(z_v / tau) / sum) / tau,  d = dloss/dlp
//
// A row is read from memory once, also for the gradient: it lies in the registers of one block (kPolicyVecs
// 16-byte vectors per thread), or of a cluster of up to 8 blocks that exchange their maxima and sums
// through distributed shared memory.  The next row's slice is on its way (one bulk copy into
// shared memory) while the current one is worked on.
//
// The partition of a row follows from the vocabulary and the type alone: a thread's elements are the same
// whatever the row's address and stride, so a row's log-probability has the same bits in every
// batch, in a strided view or a dense tensor, in the forward and with the gradient.  A ratio between
// a rollout and a trainer that saw the same logits is then exactly 1.
#pragma once

#include "layer_common.cuh"
#include "tma.cuh"

namespace gdn {

constexpr int kPolicyVecs = 8;         // 16-byte vectors of a row per thread
constexpr int kPolicyMaxThreads = 1024;
constexpr int kPolicyMaxCluster = 8;
// the largest row: a cluster's registers
constexpr int64_t kPolicyMaxBytes = (int64_t)kPolicyMaxCluster * kPolicyMaxThreads * kPolicyVecs * 16;

struct PolicyArgs {
    const void* z;
    int64_t ldz;
    const int64_t* y;
    const float *old, *ref, *adv, *dloss;  // old == null: log-probabilities only
    float lo, hi, kl;                      // borders of the ratio, weight of the KL term
    float c, inv_tau;                      // log2(e) / tau, 1 / tau
    int64_t T;
    int32_t V, slice;                      // elements of a row, and of a block of its cluster
    float *loss, *lp;
    void* dz;
    int32_t* status;
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(const void* local, uint32_t rank, float v)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
// n bytes, a multiple of 16, both addresses 16-byte aligned
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)), "l"(src), "r"(n), "r"(smem_addr(mbar))
                 : "memory");
}

// The 16 bytes that start s bytes into the 32 bytes a, b (s below 16, the same for the whole block).
__device__ __forceinline__ uint4 bytes_at(const uint4& a, const uint4& b, int s)
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t v[5];
    const int n = s >> 2;
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = n == 0 ? w[i] : n == 1 ? w[i + 1] : n == 2 ? w[i + 2] : w[i + 3];
    const int sh = (s & 3) * 8;
    return make_uint4(__funnelshift_r(v[0], v[1], sh), __funnelshift_r(v[1], v[2], sh),
                      __funnelshift_r(v[2], v[3], sh), __funnelshift_r(v[3], v[4], sh));
}

// maxima of -inf (nothing yet, or nothing but -inf) count as 0 where they are taken off an exponent
__device__ __forceinline__ float policy_base(float m) { return m == -INFINITY ? 0.0f : m; }

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

// The maximum and the sum of 2^(x - maximum) over a warp, from each lane's own; the same in every lane.
__device__ __forceinline__ void policy_warp(float& m, float& sum)
{
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
    sum *= ex2(m - policy_base(M));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    m = M;
}

// ALIGNED: every row of the logits and of the gradient is whole 16-byte vectors.
template <typename T, bool BWD, bool ALIGNED>
__global__ void __launch_bounds__(kPolicyMaxThreads, 1) k_policy(const PolicyArgs a)
{
    constexpr int E = 16 / (int)sizeof(T);  // elements of a vector
    constexpr int NV = kPolicyVecs;
    extern __shared__ __align__(128) unsigned char policy_smem[];  // the slice at its global address mod 16
    __shared__ __align__(8) uint64_t bar;
    __shared__ float wm[32], ws[32], target_logit;      // maxima and sums of the warps
    __shared__ float peer[2][kPolicyMaxCluster][3];     // of the cluster's blocks, and the target's logit; by row parity
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const int64_t first = blockIdx.x / blocks, step = gridDim.x / blocks;
    const int tid = threadIdx.x, NT = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int lo = min((int)rank * a.slice, a.V), len = min(a.slice, a.V - lo);  // this block's elements; the last may have none
    const int nvec = (len + E - 1) / E;
    if (tid == 0) mbar_init_cta(&bar, 1);
    __syncthreads();

    auto target = [&](int64_t row) -> int64_t {  // -1: a row that takes no part
        if (row >= a.T) return -1;
        const int64_t y = a.y[row];
        if (y >= a.V && tid == 0 && rank == 0 && a.status != nullptr) atomicCAS(a.status, GDN_OK, GDN_ERR_DEVICE_INPUT);
        return y >= a.V || y < 0 ? -1 : y;
    };
    // The slice's 16-byte granules in one copy; the up to 2 (E - 1) elements around them by threads 0 .. 2 E - 1.
    auto place = [&](int64_t row, int& s, int& head, int& body) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.z) + row * a.ldz + lo);
        s = ALIGNED ? 0 : (int)(p & 15);
        head = s ? min(len, (16 - s) / (int)sizeof(T)) : 0;
        body = (len - head) / E * E;
    };
    T edge{};  // an element that the copy does not cover
    const int issuer = NT - 32;  // a thread of the last warp
    auto issue = [&](int64_t row) {
        int s, head, body;
        place(row, s, head, body);
        const T* src = static_cast<const T*>(a.z) + row * a.ldz + lo;
        if constexpr (!ALIGNED) {
            if (tid < E) {
                if (tid < head) edge = src[tid];
            } else if (tid < 2 * E) {
                if (head + body + tid - E < len) edge = src[head + body + tid - E];
            }
        }
        if (tid == issuer) {
            mbar_arrive_expect_tx(&bar, (uint32_t)(body * sizeof(T)));
            if (body > 0) bulk_load(policy_smem + s + head * sizeof(T), src + head, (uint32_t)(body * sizeof(T)), &bar);
        }
    };

    int64_t y = target(first), y_next = target(first + step);
    if (y >= 0) issue(first);
    uint32_t parity = 0;
    int turn = 0;
    bool lost = false;
    for (int64_t row = first; row < a.T; row += step) {
        const int64_t y_after = target(row + 2 * step);
        if (y < 0) {  // nothing read, no exchange; the same in every block of the cluster
            if (rank == 0 && tid == 0) {
                if (a.loss != nullptr) a.loss[row] = 0.0f;
                if (a.lp != nullptr) a.lp[row] = 0.0f;
            }
            if constexpr (BWD) {
                T* out = static_cast<T*>(a.dz) + row * a.V + lo;
                if constexpr (ALIGNED) {
                    for (int i = tid; i < nvec; i += NT) *reinterpret_cast<uint4*>(out + i * E) = make_uint4(0, 0, 0, 0);
                } else {
                    for (int i = tid; i < len; i += NT) out[i] = from_f<T>(0.0f);
                }
            }
            if (y_next >= 0 && !lost) issue(row + step);
            y = y_next, y_next = y_after;
            continue;
        }
        // what the row's end needs, on its way from here on
        const float old = a.old != nullptr ? a.old[row] : 0.0f, adv = a.old != nullptr ? a.adv[row] : 0.0f;
        const float ref = a.ref != nullptr ? a.ref[row] : 0.0f, dloss = BWD ? a.dloss[row] : 0.0f;
        int s = 0;
        if constexpr (!ALIGNED) {
            int head, body;
            place(row, s, head, body);
            T* at = reinterpret_cast<T*>(policy_smem + s);
            if (tid < E) {
                if (tid < head) at[tid] = edge;
            } else if (tid < 2 * E) {
                if (head + body + tid - E < len) at[head + body + tid - E] = edge;
            } else if (tid < 3 * E) {  // the last vector is filled up with -inf
                if (len + tid - 2 * E < nvec * E) at[len + tid - 2 * E] = from_f<T>(-INFINITY);
            }
            __syncthreads();
        }
        if (!lost && !mbar_wait_bounded(&bar, parity, 1ll << 31)) lost = true;
        parity ^= 1;

        // this thread's vectors, packed
        Vec<T, E> v[NV];
        PolicyMax<T, E> top;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = tid + j * NT;
            if (i < nvec) {
                const uint4* p = reinterpret_cast<const uint4*>(policy_smem) + i;
                uint4 r = p[0];
                if (!ALIGNED && s != 0) r = bytes_at(r, p[1], s);
                v[j] = *reinterpret_cast<const Vec<T, E>*>(&r);
                top.add(v[j]);
            }
        }
        if (tid == 0 && y >= lo && y < lo + len) target_logit = to_f<T>(reinterpret_cast<const T*>(policy_smem + s)[y - lo]);
        const f2x c2 = pk2(a.c, a.c);
        float m = top.get() * a.c, sum;  // in units of log2 from here on
        {
            const float base = -policy_base(m);
            const f2x b2 = pk2(base, base);
            f2x s0 = pk2(0.0f, 0.0f), s1 = s0;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (tid + j * NT < nvec) {
#pragma unroll
                    for (int k = 0; k < E / 2; ++k) {
                        float x0, x1;
                        up2(pfma(pbits<T, E>(v[j], k), c2, b2), x0, x1);
                        f2x& acc = k & 1 ? s1 : s0;
                        acc = padd(acc, pk2(ex2(x0), ex2(x1)));
                    }
                }
            sum = psum(padd(s0, s1));
        }
        policy_warp(m, sum);
        if (lane == 0) wm[warp] = m, ws[warp] = sum;
        fence_proxy_async_smem();
        __syncthreads();  // also: the slice is in registers
        if (y_next >= 0 && !lost) issue(row + step);
        if (warp == 0) {
            m = lane < NT / 32 ? wm[lane] : -INFINITY;
            sum = lane < NT / 32 ? ws[lane] : 0.0f;
            policy_warp(m, sum);
            if (lane < (int)blocks) {
                st_cluster(&peer[turn][rank][0], lane, m);
                st_cluster(&peer[turn][rank][1], lane, sum);
                st_cluster(&peer[turn][rank][2], lane, target_logit);
            }
        }
        cluster_sync();  // also this block's barrier: a slot of this parity is written again two exchanges later
        m = peer[turn][0][0];
        for (uint32_t b = 1; b < blocks; ++b) m = fmaxf(m, peer[turn][b][0]);
        const float bm = policy_base(m);
        sum = 0.0f;
        for (uint32_t b = 0; b < blocks; ++b) sum = __fmaf_rn(peer[turn][b][1], ex2(peer[turn][b][0] - bm), sum);
        const float zy = peer[turn][(uint32_t)y / (uint32_t)a.slice][2];
        turn ^= 1;
        const float lp = (__fmaf_rn(zy, a.c, -bm) - log2f(sum)) * 0.69314718055994530942f;
        float loss = 0.0f, d = 0.0f;
        if (a.old != nullptr) {
            const float ratio = ex2((lp - old) * kLog2e);
            if (adv != 0.0f) {  // a zero takes no part, whatever the ratio
                const float free = -adv * ratio, held = -adv * fminf(fmaxf(ratio, a.lo), a.hi);
                loss = free < held ? held : free;  // not a number where the ratio is not
                d = free < held ? 0.0f : free;
            }
            if (a.ref != nullptr) {
                const float gap = ref - lp, e = ex2(gap * kLog2e);
                loss = __fmaf_rn(a.kl, e - gap - 1.0f, loss);
                d = __fmaf_rn(a.kl, 1.0f - e, d);
            }
        }
        if (rank == 0 && tid == 0) {
            if (a.loss != nullptr) a.loss[row] = loss;
            if (a.lp != nullptr) a.lp[row] = lp;
        }
        if constexpr (BWD) {
            d *= dloss * a.inv_tau;
            const float scale = -d / sum;
            const f2x b2 = pk2(-bm, -bm), scale2 = pk2(scale, scale);
            T* out = static_cast<T*>(a.dz) + row * a.V + lo;
            const int so = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(out) & 15);
            const int yl = (int)y - lo;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = tid + j * NT;
                if (i - lane < nvec && !lost) {  // the whole warp: it exchanges below
                    f2x o[E / 2];
#pragma unroll
                    for (int k = 0; k < E / 2; ++k) {
                        float x0, x1;
                        up2(pfma(pbits<T, E>(v[j], k), c2, b2), x0, x1);
                        o[k] = pmul(pk2(ex2(x0), ex2(x1)), scale2);
                    }
                    if ((unsigned)(yl - i * E) < (unsigned)E) {
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) {
                            const int q = yl - i * E - 2 * k;
                            o[k] = padd(o[k], pk2(q == 0 ? d : 0.0f, q == 1 ? d : 0.0f));
                        }
                    }
                    if constexpr (ALIGNED) {
                        if (i < nvec) pstore<T, E>(out + i * E, o);
                    } else {
                        // The rows start anywhere: a thread stores the 16 bytes of memory that begin in its
                        // neighbour's vector and end in its own.  The warp's first and last bytes, and the row's, go one by one.
                        Vec<T, E> r;
                        pstore<T, E>(r.v, o);
                        const uint4 own = *reinterpret_cast<const uint4*>(&r);
                        uint4 left;
                        left.x = __shfl_up_sync(kFullMask, own.x, 1);
                        left.y = __shfl_up_sync(kFullMask, own.y, 1);
                        left.z = __shfl_up_sync(kFullMask, own.z, 1);
                        left.w = __shfl_up_sync(kFullMask, own.w, 1);
                        const int cut = so / (int)sizeof(T);  // elements of a vector that belong to the next 16 bytes
                        auto fits = [&](int i) { return i < nvec && i * E + E - cut <= len; };
                        const bool joined = fits(i) && (lane > 0 || cut == 0);
                        if (joined) *reinterpret_cast<uint4*>(out + i * E - cut) = cut == 0 ? own : bytes_at(left, own, 16 - so);
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            const bool mine = k < E - cut ? !joined : lane == 31 || !fits(i + 1);
                            if (i < nvec && mine && i * E + k < len) out[i * E + k] = r.v[k];
                        }
                    }
                }
            }
        }
        y = y_next, y_next = y_after;
    }
    if (lost) {
        if (a.status != nullptr) atomicCAS(a.status, GDN_OK, GDN_ERR_TIMEOUT);
        mbar_wait_bounded(&bar, parity ^ 1, 1ll << 31);  // the copy that was late
    }
}

}  // namespace gdn

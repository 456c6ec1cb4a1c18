// k_qknorm.cuh -- norms of the queries' and keys' heads with the position rotation in the same
// pass, forward and backward (sm_100a).
//
//     r = (sum x^2 / n + eps)^(-1/2),  u = x r w      (n = d, or 1 for unit length)
//     the first R dimensions turn in pairs (a, b) by the angle p f_i of the token's position p:
//     a' = a cos - b sin,  b' = b cos + a sin
// and, with g = the gradient turned back and h = g w:
//     dx = r (h - x r sum(h x) r / n),  dw = sum_rows g x r
//
// One read of x (and dy), one write, q and k in one launch.  A row (one head of one token) lies in the
// registers of tpr neighbouring lanes, each with four pairs, so that a pair's two elements meet in one
// thread and turn without an exchange.  A block takes `tokens` tokens at a time and
// makes their angles once, for all heads, in shared memory: position times frequency in turns
// and in 64 bits, so that far positions keep their angle (at 10^6 tokens fp32 is off by 0.06), with the whole turns
// taken off before sincospi in fp32.
#pragma once

#include "layer_common.cuh"
#include "k_norm.cuh"

namespace gdn {

struct QkArgs {
    const void* x[2];   // q, k
    int64_t ldx[2];
    const void* dy[2];  // backward: gradients of the outputs
    int64_t lddy[2];
    void* out[2];       // the outputs, or the gradients of the inputs
    const void* w[2];
    int32_t H[2];
    int32_t w_bf16, interleaved;
    const int32_t* pos;
    const float* freq;
    float eps, inv_n;
    int64_t T;
    int32_t d, rot, tpr;
    int32_t tokens;     // per tile
    float* part;        // backward: [grid][2][d] sums of dw, or null
};

constexpr int kQkThreads = 256;
__host__ __device__ constexpr int qk_rows(bool bwd) { return bwd ? 2 : 4; }  // rows of a thread in flight

// The elements of a thread's pair i (of 4 neighbouring ones).
template <bool VEC>
struct QkPairs {
    int first, n, R2, inter;
    __device__ __forceinline__ QkPairs(const QkArgs& a, int lane)
        : first(lane * 4), n(a.d / 2), R2(a.rot / 2), inter(a.interleaved) {}
    __device__ __forceinline__ int pair(int i) const { return first + i; }
    __device__ __forceinline__ bool has(int i) const { return (VEC ? first : first + i) < n; }  // VEC: all four or none
    // the pair's two elements; behind the rotated ones any two that are left
    __device__ __forceinline__ int a(int i) const
    {
        const int p = pair(i);
        return inter ? 2 * p : (p < R2 ? p : p + R2);
    }
    __device__ __forceinline__ int b(int i) const
    {
        const int p = pair(i);
        return inter ? 2 * p + 1 : (p < R2 ? p + R2 : p + n);
    }
};

// A thread's share of a row: va and vb hold the elements a and b of its four pairs.  VEC: two accesses of
// four elements, else one element at a time; the sums, and with them the bits, are the same.
template <typename T, bool VEC>
struct QkRow {
    Vec<T, 4> lo, hi;
    __device__ __forceinline__ void load(const T* row, const QkPairs<VEC>& q)
    {
        if constexpr (VEC) {
            if (q.has(0)) {
                lo = load_vec<T, 4>(row + q.a(0));
                hi = load_vec<T, 4>(row + (q.inter ? q.a(2) : q.b(0)));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q.has(i)) {
                    lo.v[i] = row[q.a(i)];
                    hi.v[i] = row[q.b(i)];
                }
        }
    }
    __device__ __forceinline__ void get(const QkPairs<VEC>& q, float (&va)[4], float (&vb)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            va[i] = q.has(i) ? to_f<T>(lo.v[i]) : 0.0f;
            vb[i] = q.has(i) ? to_f<T>(hi.v[i]) : 0.0f;
        }
        if (VEC && q.inter) swap(va, vb);
    }
    // neighbouring pairs: (a0 b0 a1 b1), (a2 b2 a3 b3) <-> (a0 a1 a2 a3), (b0 b1 b2 b3)
    __device__ static __forceinline__ void swap(float (&va)[4], float (&vb)[4])
    {
        const float x1 = va[1], x2 = va[2], x3 = va[3], y0 = vb[0], y1 = vb[1], y2 = vb[2];
        va[1] = x2, va[2] = y0, va[3] = y2;
        vb[0] = x1, vb[1] = x3, vb[2] = y1;
    }
    __device__ static __forceinline__ void join(float (&va)[4], float (&vb)[4])
    {
        const float a1 = va[1], a2 = va[2], a3 = va[3], b0 = vb[0], b1 = vb[1], b2 = vb[2];
        va[1] = b0, va[2] = a1, va[3] = b1;
        vb[0] = a2, vb[1] = b2, vb[2] = a3;
    }
    __device__ static __forceinline__ void store(T* row, const QkPairs<VEC>& q, float (&va)[4], float (&vb)[4])
    {
        if constexpr (VEC) {
            if (q.has(0)) {
                if (q.inter) join(va, vb);
                store_vec<T, 4>(row + q.a(0), va);
                store_vec<T, 4>(row + (q.inter ? q.a(2) : q.b(0)), vb);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q.has(i)) {
                    row[q.a(i)] = from_f<T>(va[i]);
                    row[q.b(i)] = from_f<T>(vb[i]);
                }
        }
    }
};

// Turns the pairs by the token's angles (sign = -1: back).
template <bool VEC>
__device__ __forceinline__ void qk_turn(const float2* cs, const QkPairs<VEC>& q, float sign, float (&va)[4], float (&vb)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (q.pair(i) < q.R2) {
            const float2 c = cs[q.pair(i)];
            const float s = c.y * sign, x = va[i], y = vb[i];
            va[i] = __fmaf_rn(x, c.x, -(y * s));
            vb[i] = __fmaf_rn(y, c.x, x * s);
        }
}

// BWD: the gradients.  T tokens, VEC as QkPairs.
template <typename T, bool VEC, bool BWD>
__global__ void __launch_bounds__(kQkThreads, BWD ? 2 : 3) k_qk_norm(const QkArgs a)
{
    constexpr int U = qk_rows(BWD);
    extern __shared__ __align__(16) unsigned char qk_smem[];
    float2* cs = reinterpret_cast<float2*>(qk_smem);                         // [tokens][rot / 2]
    float* ws = reinterpret_cast<float*>(cs + (int64_t)a.tokens * (a.rot / 2));  // [2][d]: the a's of all pairs, then the b's
    const int tpr = a.tpr, lane = threadIdx.x & (tpr - 1), slot = threadIdx.x / tpr, slots = kQkThreads / tpr;
    const int n = a.d / 2, R2 = a.rot / 2;
    const QkPairs<VEC> pairs(a, lane);
    for (int i = threadIdx.x; i < 2 * a.d; i += kQkThreads) {
        const int kind = i / a.d, e = i % a.d, p = e < n ? e : e - n;
        const int at = a.interleaved ? 2 * p + (e >= n) : (e < n ? (p < R2 ? p : p + R2) : (p < R2 ? p + R2 : p + n));
        ws[i] = a.w[kind] != nullptr ? load_w(a.w[kind], a.w_bf16, at) : 1.0f;
    }
    __syncthreads();
    float da[2][4], db[2][4];  // backward: this thread's columns of dw, of q and k
#pragma unroll
    for (int i = 0; i < 4; ++i) da[0][i] = da[1][i] = db[0][i] = db[1][i] = 0.0f;

    const int64_t tiles = (a.T + a.tokens - 1) / a.tokens;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t t0 = tile * a.tokens;
        const int nt = (int)min((int64_t)a.tokens, a.T - t0);
        if (R2 > 0) {
            __syncthreads();  // the last tile's angles have been read
            for (int i = threadIdx.x; i < nt * R2; i += kQkThreads) {
                const int t = i / R2, p = i - t * R2;
                const double turns = (double)a.pos[t0 + t] * ((double)a.freq[p] * 0.15915494309189533577);
                float s, c;
                sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
                cs[i] = make_float2(c, s);
            }
            __syncthreads();
        }
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const int H = a.H[kind], rows = nt * H;
            const T* x0 = static_cast<const T*>(a.x[kind]) + t0 * a.ldx[kind];
            const T* g0 = BWD ? static_cast<const T*>(a.dy[kind]) + t0 * a.lddy[kind] : nullptr;
            T* o0 = static_cast<T*>(a.out[kind]) + t0 * H * a.d;
            float wa[4], wb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wa[i] = pairs.has(i) ? ws[kind * a.d + pairs.pair(i)] : 0.0f;
                wb[i] = pairs.has(i) ? ws[kind * a.d + n + pairs.pair(i)] : 0.0f;
            }
            for (int r0 = 0; r0 < rows; r0 += slots * U) {  // the same turns for every thread: the sums are shuffles
                QkRow<T, VEC> x[U], g[BWD ? U : 1];
                int tok[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * slots + slot;
                    tok[u] = r / H;
                    if (r < rows) {
                        x[u].load(x0 + tok[u] * a.ldx[kind] + (r - tok[u] * H) * a.d, pairs);
                        if constexpr (BWD) g[u].load(g0 + tok[u] * a.lddy[kind] + (r - tok[u] * H) * a.d, pairs);
                    }
                }
                float ss[U], sg[BWD ? U : 1];
                float ga[BWD ? U : 1][4], gb[BWD ? U : 1][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool on = r0 + u * slots + slot < rows;
                    float va[4], vb[4];
                    x[u].get(pairs, va, vb);
                    ss[u] = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) ss[u] = __fmaf_rn(va[i], va[i], __fmaf_rn(vb[i], vb[i], ss[u]));
                    if constexpr (BWD) {
                        sg[u] = 0.0f;
                        if (on) {
                            g[u].get(pairs, ga[u], gb[u]);
                            qk_turn<VEC>(cs + tok[u] * R2, pairs, -1.0f, ga[u], gb[u]);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sg[u] = __fmaf_rn(ga[u][i] * wa[i], va[i], __fmaf_rn(gb[u][i] * wb[i], vb[i], sg[u]));
                        }
                    }
                }
                for (int o = tpr >> 1; o > 0; o >>= 1) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        ss[u] += __shfl_xor_sync(kFullMask, ss[u], o);
                        if constexpr (BWD) sg[u] += __shfl_xor_sync(kFullMask, sg[u], o);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * slots + slot;
                    if (r >= rows) continue;
                    const float rr = inv_sqrt(__fmaf_rn(ss[u], a.inv_n, a.eps));
                    float va[4], vb[4];
                    x[u].get(pairs, va, vb);
                    if constexpr (BWD) {
                        // as in layer norm, no power of r is formed: x r is again about 1
                        const float c = sg[u] * rr * a.inv_n;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float na = va[i] * rr, nb = vb[i] * rr;
                            da[kind][i] = __fmaf_rn(ga[u][i], na, da[kind][i]);
                            db[kind][i] = __fmaf_rn(gb[u][i], nb, db[kind][i]);
                            va[i] = rr * __fmaf_rn(-na, c, ga[u][i] * wa[i]);
                            vb[i] = rr * __fmaf_rn(-nb, c, gb[u][i] * wb[i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            va[i] = va[i] * rr * wa[i];
                            vb[i] = vb[i] * rr * wb[i];
                        }
                        qk_turn<VEC>(cs + tok[u] * R2, pairs, 1.0f, va, vb);
                    }
                    QkRow<T, VEC>::store(o0 + (int64_t)r * a.d, pairs, va, vb);
                }
            }
        }
    }
    if (!BWD || a.part == nullptr) return;
    // dw: the rows of a warp by shuffles, then the warps in order
    float* red = ws;  // [8][d], behind the angles; the weights are in registers
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        for (int o = 16; o >= tpr; o >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                da[kind][i] += __shfl_xor_sync(kFullMask, da[kind][i], o);
                db[kind][i] += __shfl_xor_sync(kFullMask, db[kind][i], o);
            }
        __syncthreads();
        if ((threadIdx.x & 31) < tpr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (pairs.has(i)) {
                    red[(threadIdx.x >> 5) * a.d + pairs.a(i)] = da[kind][i];
                    red[(threadIdx.x >> 5) * a.d + pairs.b(i)] = db[kind][i];
                }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kQkThreads) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kQkThreads / 32; ++w) s += red[w * a.d + c];
            part[kind * a.d + c] = s;
        }
    }
}

// [2][d] column sums -> the gradients of the two weights
struct QkGradMap {
    float *q, *k;
    int32_t d;
    __device__ void operator()(int64_t m, float s) const
    {
        if (m < d) {
            if (q != nullptr) q[m] = s;
        } else if (k != nullptr) {
            k[m - d] = s;
        }
    }
};

}  // namespace gdn

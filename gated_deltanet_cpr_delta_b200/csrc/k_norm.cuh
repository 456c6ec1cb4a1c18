// k_norm.cuh -- layer norm over the last axis, forward and backward (sm_100a).
//
//     mean = sum x / D,  rstd = (sum (x - mean)^2 / D + eps)^(-1/2)
//     n = (x - mean) rstd,  y = n w + b
// and with g = dy w:
//     dx = rstd (g - sum g / D - n sum(g n) / D),  dw = sum_rows dy n,  db = sum_rows dy
//
// Bound by memory: one read of x (and dy), one write.  A row stays in the
// registers of `tpr` threads (NV vectors of V elements each), so the variance
// is the second moment about the mean, exact to fp32 also for rows whose mean
// is large, without a second read.
#pragma once

#include "layer_common.cuh"

namespace gdn {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormBwdThreads = 512;

struct NormArgs {
    const void* x;
    int64_t ldx;
    const void* dy;
    int64_t lddy;
    const void *w, *b;
    int w_bf16;
    float eps;
    int64_t R;
    int32_t D;
    int32_t tpr;  // threads per row: a power of two up to the block's size
    void *y, *dx;
    float *mean, *rstd, *part;
};

// Sums of K values over the tpr threads of a row; red: [K][32] floats of this
// block, used when a row spans warps.  Every thread of the block calls it.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o < tpr) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(kFullMask, v[k], o);
        }
    }
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, wpr = tpr >> 5, first = warp & ~(wpr - 1);
        __syncthreads();  // the previous sums have been read
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[k * 32 + warp] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
            for (int i = 0; i < wpr; ++i) s += red[k * 32 + first + i];
            v[k] = s;
        }
    }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kNormMaxThreads) k_norm_fwd(const NormArgs a)
{
    __shared__ float red[32];
    const int rpb = blockDim.x / a.tpr;
    const int lane = threadIdx.x & (a.tpr - 1);
    const int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / a.tpr;
    const bool on = row < a.R;
    const T* x = static_cast<const T*>(a.x) + (on ? row : 0) * a.ldx;
    float v[NV][V];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * a.tpr + lane) * V;
        if (on && c < a.D) {
            const Vec<T, V> r = load_vec<T, V>(x + c);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                v[i][k] = to_f<T>(r.v[k]);
                s[0] += v[i][k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) v[i][k] = 0.0f;
        }
    }
    row_sum<1>(s, a.tpr, red);
    const float mean = s[0] / (float)a.D;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((i * a.tpr + lane) * V < a.D) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                v[i][k] -= mean;
                s[0] = __fmaf_rn(v[i][k], v[i][k], s[0]);
            }
        }
    }
    row_sum<1>(s, a.tpr, red);
    const float rstd = 1.0f / sqrtf(s[0] / (float)a.D + a.eps);
    if (!on) return;
    T* y = static_cast<T*>(a.y) + row * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * a.tpr + lane) * V;
        if (c < a.D) {
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float n = v[i][k] * rstd;
                o[k] = a.b != nullptr ? __fmaf_rn(n, load_w(a.w, a.w_bf16, c + k), load_w(a.b, a.w_bf16, c + k))
                                      : n * load_w(a.w, a.w_bf16, c + k);
            }
            store_vec<T, V>(y + c, o);
        }
    }
    if (lane == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

// Rows too wide for the registers of a block: one block per row, which reads
// the row three times (from L2 after the first).
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_fwd_wide(const NormArgs a)
{
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.y) + row * a.D;
    float s[1] = {0.0f};
    for (int c = threadIdx.x; c < a.D; c += 1024) s[0] += to_f<T>(x[c]);
    row_sum<1>(s, 1024, red);
    const float mean = s[0] / (float)a.D;
    s[0] = 0.0f;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float d = to_f<T>(x[c]) - mean;
        s[0] = __fmaf_rn(d, d, s[0]);
    }
    row_sum<1>(s, 1024, red);
    const float rstd = 1.0f / sqrtf(s[0] / (float)a.D + a.eps);
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float n = (to_f<T>(x[c]) - mean) * rstd, w = load_w(a.w, a.w_bf16, c);
        y[c] = from_f<T>(a.b != nullptr ? __fmaf_rn(n, w, load_w(a.b, a.w_bf16, c)) : n * w);
    }
    if (threadIdx.x == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

// Each block walks rows with a stride and keeps its share of dw and db in
// registers: a thread's columns are the same in every row.  The shares of the
// blocks ([grid][2][D]) are joined by k_colsum.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kNormBwdThreads) k_norm_bwd(const NormArgs a)
{
    extern __shared__ float sh[];  // [64] row sums, then [2][D] when several rows share a block
    float* red = sh;
    const int rpb = blockDim.x / a.tpr;
    const int lane = threadIdx.x & (a.tpr - 1), sub = threadIdx.x / a.tpr;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (i * a.tpr + lane) * V + k;
            w[i][k] = c < a.D ? load_w(a.w, a.w_bf16, c) : 0.0f;
            dw[i][k] = db[i][k] = 0.0f;
        }
    const float inv = 1.0f / (float)a.D;
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.R; r0 += (int64_t)gridDim.x * rpb) {
        const int64_t row = r0 + sub;
        const bool on = row < a.R;
        const T* x = static_cast<const T*>(a.x) + (on ? row : 0) * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + (on ? row : 0) * a.lddy;
        const float mean = on ? a.mean[row] : 0.0f, rstd = on ? a.rstd[row] : 0.0f;
        float n[NV][V], g[NV][V];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * a.tpr + lane) * V;
            if (on && c < a.D) {
                const Vec<T, V> rx = load_vec<T, V>(x + c), rg = load_vec<T, V>(dy + c);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    n[i][k] = (to_f<T>(rx.v[k]) - mean) * rstd;
                    const float d = to_f<T>(rg.v[k]);
                    dw[i][k] = __fmaf_rn(d, n[i][k], dw[i][k]);
                    db[i][k] += d;
                    g[i][k] = d * w[i][k];
                    s[0] += g[i][k];
                    s[1] = __fmaf_rn(g[i][k], n[i][k], s[1]);
                }
            }
        }
        row_sum<2>(s, a.tpr, red);
        const float mg = s[0] * inv, mgn = s[1] * inv;
        if (on) {
            T* dx = static_cast<T*>(a.dx) + row * a.D;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * a.tpr + lane) * V;
                if (c < a.D) {
                    float o[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] = rstd * (g[i][k] - __fmaf_rn(n[i][k], mgn, mg));
                    store_vec<T, V>(dx + c, o);
                }
            }
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.D;
    if (rpb == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c = (i * a.tpr + lane) * V + k;
                if (c < a.D) {
                    part[c] = dw[i][k];
                    part[a.D + c] = db[i][k];
                }
            }
        return;
    }
    // the rows of a block, joined one after the other (their order is fixed)
    float* acc = sh + 64;
    for (int r = 0; r < rpb; ++r) {
        __syncthreads();
        if (sub == r) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int c = (i * a.tpr + lane) * V + k;
                    if (c < a.D) {
                        acc[c] = (r ? acc[c] : 0.0f) + dw[i][k];
                        acc[a.D + c] = (r ? acc[a.D + c] : 0.0f) + db[i][k];
                    }
                }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += blockDim.x) part[c] = acc[c];
}

// Wide rows: one block per row for dx (two reads of the row); dw and db by columns.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_bwd_wide(const NormArgs a)
{
    __shared__ float red[64];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    T* dx = static_cast<T*>(a.dx) + row * a.D;
    const float mean = a.mean[row], rstd = a.rstd[row], inv = 1.0f / (float)a.D;
    float s[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float g = to_f<T>(dy[c]) * load_w(a.w, a.w_bf16, c);
        s[0] += g;
        s[1] = __fmaf_rn(g, (to_f<T>(x[c]) - mean) * rstd, s[1]);
    }
    row_sum<2>(s, 1024, red);
    const float mg = s[0] * inv, mgn = s[1] * inv;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float n = (to_f<T>(x[c]) - mean) * rstd;
        dx[c] = from_f<T>(rstd * (to_f<T>(dy[c]) * load_w(a.w, a.w_bf16, c) - __fmaf_rn(n, mgn, mg)));
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_norm_bwd_wide_w(const NormArgs a)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < a.R; r += gridDim.y) {
        const float d = to_f<T>(static_cast<const T*>(a.dy)[r * a.lddy + c]);
        dw = __fmaf_rn(d, (to_f<T>(static_cast<const T*>(a.x)[r * a.ldx + c]) - a.mean[r]) * a.rstd[r], dw);
        db += d;
    }
    a.part[(int64_t)blockIdx.y * 2 * a.D + c] = dw;
    a.part[(int64_t)blockIdx.y * 2 * a.D + a.D + c] = db;
}

// [2][D] column sums -> dweight, dbias
struct NormGradMap {
    float *dw, *db;
    int32_t D;
    __device__ void operator()(int64_t m, float s) const
    {
        if (m < D) dw[m] = s;
        else if (db != nullptr) db[m - D] = s;
    }
};

}  // namespace gdn

// k_norm.cuh -- layer norm over the last axis, forward and backward (sm_100a).
//
//     mean = sum x / D,  rstd = (sum (x - mean)^2 / D + eps)^(-1/2)
//     n = (x - mean) rstd,  y = n w + b
// and with g = dy w:
//     dx = rstd (g - sum g / D - n sum(g n) / D),  dw = sum_rows dy n,  db = sum_rows dy
//
// One read of x (and dy), one write; bound by the latency of memory and of the rows' sums, with DRAM at
// 43% (forward) and 58% of its peak.  A row stays in the
// registers of `tpr` threads (NV vectors of V elements each), so the variance
// is the second moment about the mean, exact to fp32 also for rows whose mean
// is large, without a second read.  Measured on a B200 (bf16): 16384 x 4096 forward
// 59 us, 4.5 TB/s, gradients 78 us, 5.2 TB/s, + 5 us for the sums of dw and db;
// 262144 rows of 128 30 us, 4.5 TB/s (there a row's two sums over 16 lanes
// bind it as much as the memory); 64 x 4096 3.5 us.  Dense rows of odd widths are read
// in 16-byte vectors that start off the row (SHIFT): 8192 x 4097 forward 60 us, gradients 85 us,
// 82 of them in k_norm_bwd (8192 x 4096: 30, 52 and 47 us; element by element 164 and 154 us).
#pragma once

#include "layer_common.cuh"

namespace gdn {


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
    auto fold = [&](int o) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(kFullMask, v[k], o);
    };
    if (tpr >= 32) fold(16);
    if (tpr >= 16) fold(8);
    fold(4);  // a row has at least 8 threads
    fold(2);
    fold(1);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, wpr = tpr >> 5, first = warp & ~(wpr - 1);
        __syncthreads();  // the previous sums have been read
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[k * 32 + warp] = v[k];
        }
        __syncthreads();
        // every warp sums the row's warps itself, wpr (2 to 32) neighbouring lanes at a time
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = red[k * 32 + first + (threadIdx.x & (wpr - 1))];
        if (wpr > 16) fold(16);
        if (wpr > 8) fold(8);
        if (wpr > 4) fold(4);
        if (wpr > 2) fold(2);
        fold(1);
    }
}

// V elements of a weight or bias, as they are stored
template <typename WT, int V>
__device__ __forceinline__ Vec<WT, V> norm_weight(const void* w, int c)
{
    const WT* p = static_cast<const WT*>(w) + c;
    Vec<WT, V> r;
    if (V > 1 && (reinterpret_cast<uintptr_t>(p) & (sizeof(r) < 16 ? sizeof(r) - 1 : 15)) == 0) {
        constexpr int E = sizeof(r) > 16 ? 16 / sizeof(WT) : V;  // elements per access
#pragma unroll
        for (int i = 0; i < V / E; ++i) {
            const Vec<WT, E> q = load_vec<WT, E>(p + i * E);
#pragma unroll
            for (int k = 0; k < E; ++k) r.v[i * E + k] = q.v[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) r.v[k] = p[k];
    }
    return r;
}

__host__ __device__ constexpr int norm_threads(int V) { return V == 1 ? 1024 : 512; }  // most threads of a block

// x^(-1/2): the approximate instruction and one step of Newton's method
__device__ __forceinline__ float inv_sqrt(float x)
{
    const float r = rsqrtf(x);
    const float e = __fmaf_rn(-x * r, r, 1.0f);  // 1 - x r^2
    return x > 0.0f && x < 3.0e38f ? __fmaf_rn(0.5f * e, r, r) : r;
}

// Keeps r packed: without it the compiler widens the weights once, before the loop
// over the rows, into twice the registers.
template <typename WT, int V>
__device__ __forceinline__ void keep_packed(Vec<WT, V>& r)
{
    if constexpr (sizeof(r) % 4 == 0) {
        uint32_t* u = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < (int)sizeof(r) / 4; ++i) asm volatile("" : "+r"(u[i]));
    }
}

// A thread's own vectors of the rows that it will work on next, in a ring in shared
// memory that cp.async fills: memory stays busy through the sums of the current row, at no cost
// in registers, and since a thread reads only what it has copied itself, the ring needs no
// barrier.  (Prefetching into registers instead left half the threads and was
// slower than no prefetch: 131 us against 95 at 16384 x 4096.)
template <typename T, int V, int NV, int DEP>
struct NormRing {
    static constexpr bool ON = V * sizeof(T) == 16;
    static constexpr size_t BYTES = ON ? (size_t)DEP * NV * 16 : 0;  // per thread and tensor
    unsigned char* base;
    __device__ __forceinline__ unsigned char* at(int slot, int i) const
    {
        return base + ((slot * NV + i) * blockDim.x + threadIdx.x) * 16u;
    }
    __device__ __forceinline__ void copy(int slot, int i, const T* src) const
    {
        if constexpr (ON)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             (unsigned)__cvta_generic_to_shared(at(slot, i))), "l"(src) : "memory");
    }
    // the first n elements; zeros behind them
    __device__ __forceinline__ void copy(int slot, int i, const T* src, int n) const
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (unsigned)__cvta_generic_to_shared(at(slot, i))), "l"(src), "r"(n * (int)sizeof(T)) : "memory");
    }
    __device__ __forceinline__ Vec<T, V> get(int slot, int i, const T* src) const
    {
        if constexpr (ON) return *reinterpret_cast<const Vec<T, V>*>(at(slot, i));
        else return load_vec<T, V>(src);
    }
    __device__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    __device__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEP - 1) : "memory"); }
};

// Rows that are not whole 16-byte vectors (SHIFT).  Dense rows of odd widths start anywhere
// within a vector, but rows V apart start alike: with a stride of a multiple of V
// rows, a thread's vectors cover the same columns in every row.  They start m columns before the row, so
// that they are aligned; the first may hold the end of the row before (cleared), the
// last stops at the row's end.  (8192 x 4097 bf16: 60 us forward, element by element 164.)
template <typename T, int V>
struct NormCols {
    int c0, step, D;  // vector i covers the columns c0 + i step ..
    __device__ __forceinline__ int at(int i) const { return c0 + i * step; }
    __device__ __forceinline__ bool any(int i) const { return at(i) < D; }
    __device__ __forceinline__ bool whole(int i) const { return at(i) >= 0 && at(i) + V <= D; }
    __device__ __forceinline__ bool has(int i, int k) const { return at(i) + k >= 0 && at(i) + k < D; }
    __device__ __forceinline__ void clear(int i, Vec<T, V>& r) const
    {
        if (!whole(i)) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (!has(i, k)) r.v[k] = from_f<T>(0.0f);
        }
    }
    __device__ __forceinline__ void clear(int i, typename Lanes<V>::type (&v)[Lanes<V>::N]) const
    {
        if (!whole(i)) {
            if constexpr (V > 1) {
#pragma unroll
                for (int k = 0; k < V / 2; ++k) {
                    float x, y;
                    up2(v[k], x, y);
                    v[k] = pk2(has(i, 2 * k) ? x : 0.0f, has(i, 2 * k + 1) ? y : 0.0f);
                }
            }
        }
    }
    __device__ __forceinline__ void store(int i, T* p, const typename Lanes<V>::type* o) const
    {
        if (whole(i)) {
            pstore<T, V>(p, o);
        } else if constexpr (V > 1) {
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                float x, y;
                up2(o[k], x, y);
                if (has(i, 2 * k)) p[2 * k] = from_f<T>(x);
                if (has(i, 2 * k + 1)) p[2 * k + 1] = from_f<T>(y);
            }
        }
    }
    template <typename WT>
    __device__ __forceinline__ Vec<WT, V> weight(int i, const void* w) const
    {
        if (whole(i)) return norm_weight<WT, V>(w, at(i));
        Vec<WT, V> r;
#pragma unroll
        for (int k = 0; k < V; ++k) r.v[k] = has(i, k) ? static_cast<const WT*>(w)[at(i) + k] : from_f<WT>(0.0f);
        return r;
    }
};

__host__ __device__ constexpr int norm_depth(int NV) { return NV == 1 ? 4 : 2; }  // rows ahead

// Blocks walk the rows with a stride, the weights in registers.  Columns beyond D hold zeros.
template <typename T, typename WT, int V, int NV, bool SHIFT>
__global__ void __launch_bounds__(norm_threads(V)) k_norm_fwd(const NormArgs a)
{
    using L = Lanes<V>;
    using P = typename L::type;
    constexpr int DEP = norm_depth(NV);
    extern __shared__ __align__(16) unsigned char norm_smem[];
    __shared__ float red[32];
    const NormRing<T, V, NV, DEP> ring{norm_smem};
    const int rpb = blockDim.x / a.tpr;
    const int lane = threadIdx.x & (a.tpr - 1);
    const int R = (int)a.R, step = gridDim.x * rpb, first = blockIdx.x * rpb + threadIdx.x / a.tpr;  // below 2^31
    const int64_t stepx = step * a.ldx, stepy = step * (int64_t)a.D;
    const int m = SHIFT ? (int)((first * (int64_t)a.D) & (V - 1)) : 0;
    const NormCols<T, V> cols{lane * V - m, a.tpr * V, a.D};
    const T* px = static_cast<const T*>(a.x) + (lane * V - m) + first * a.ldx;  // the row to copy next
    const T* cx = px;                                                     // the row to work on
    T* py = static_cast<T*>(a.y) + (lane * V - m) + first * (int64_t)a.D;
    Vec<WT, V> w[NV], b[NV];
    auto fetch = [&](int left, int slot) {  // left: rows from this one to the last
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (cols.any(i)) {
                    if constexpr (SHIFT) ring.copy(slot, i, px + i * a.tpr * V, min(V, a.D - cols.at(i)));
                    else ring.copy(slot, i, px + i * a.tpr * V);
                }
        }
        px += stepx;
        ring.commit();
    };
    int left = R - first;  // rows from the thread's current one to the last
#pragma unroll
    for (int j = 0; j < DEP; ++j) fetch(left - j * step, j);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (cols.any(i)) {
            w[i] = cols.template weight<WT>(i, a.w);
            if (a.b != nullptr) b[i] = cols.template weight<WT>(i, a.b);
        }
    }
    const float inv = 1.0f / (float)a.D;
    int slot = 0;
    float *pm = a.mean + first, *pr = a.rstd + first;
    for (int rest = R - blockIdx.x * rpb; rest > 0;
         rest -= step, left -= step, cx += stepx, py += stepy, pm += step, pr += step) {
        const bool on = left > 0;
        P v[NV][L::N];
        P acc = pset<V>(0.0f);
        ring.wait();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = on && cols.any(i);
            Vec<T, V> r;
            if (in) r = ring.get(slot, i, cx + i * a.tpr * V);
            if (SHIFT && in) cols.clear(i, r);
#pragma unroll
            for (int k = 0; k < L::N; ++k) {
                v[i][k] = in ? pbits<T, V>(r, k) : pset<V>(0.0f);
                acc = padd(acc, v[i][k]);
            }
        }
        float s[1] = {psum(acc)};
        row_sum<1>(s, a.tpr, red);
        fetch(left - DEP * step, slot);  // behind the sum that used the slot's last row
        slot = slot + 1 == DEP ? 0 : slot + 1;
        const float mean = s[0] * inv;
        acc = pset<V>(0.0f);
        const P minus = pset<V>(-mean);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (cols.any(i)) {
#pragma unroll
                for (int k = 0; k < L::N; ++k) v[i][k] = padd(v[i][k], minus);
                if (SHIFT) cols.clear(i, v[i]);
#pragma unroll
                for (int k = 0; k < L::N; ++k) acc = pfma(v[i][k], v[i][k], acc);
            }
        }
        s[0] = psum(acc);
        row_sum<1>(s, a.tpr, red);
        const float rstd = inv_sqrt(__fmaf_rn(s[0], inv, a.eps));
        if (on) {
            const P r2 = pset<V>(rstd);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                keep_packed(w[i]);
                keep_packed(b[i]);
                if (cols.any(i)) {
                    P o[L::N];
#pragma unroll
                    for (int k = 0; k < L::N; ++k) {
                        o[k] = pmul(v[i][k], r2);
                        o[k] = a.b != nullptr ? pfma(o[k], pbits<WT, V>(w[i], k), pbits<WT, V>(b[i], k))
                                              : pmul(o[k], pbits<WT, V>(w[i], k));
                    }
                    if constexpr (SHIFT) cols.store(i, py + i * a.tpr * V, o);
                    else pstore<T, V>(py + i * a.tpr * V, o);
                }
            }
            if (lane == 0) {
                *pm = mean;
                *pr = rstd;
            }
        }
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
    const float rstd = inv_sqrt(s[0] / (float)a.D + a.eps);
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
// registers: a thread's columns are the same in every row.  The next rows and their statistics
// are on their way meanwhile.  The shares of the blocks ([grid][2][D]) are joined by k_colsum.
template <typename T, typename WT, int V, int NV, bool SHIFT>
__global__ void __launch_bounds__(512) k_norm_bwd(const NormArgs a)
{
    using L = Lanes<V>;
    using P = typename L::type;
    constexpr int DEP = norm_depth(NV);
    using Ring = NormRing<T, V, NV, DEP>;
    extern __shared__ __align__(16) unsigned char norm_smem[];  // two rings; later [2][D] when several rows share a block
    __shared__ float red[64];
    const Ring ringx{norm_smem}, ringg{norm_smem + Ring::BYTES * blockDim.x};
    const int rpb = blockDim.x / a.tpr;
    const int lane = threadIdx.x & (a.tpr - 1), sub = threadIdx.x / a.tpr;
    const int R = (int)a.R, step = gridDim.x * rpb, first = blockIdx.x * rpb + sub;  // below 2^31
    const int64_t stepx = step * a.ldx, stepg = step * a.lddy, stepd = step * (int64_t)a.D;
    const int m = SHIFT ? (int)((first * (int64_t)a.D) & (V - 1)) : 0;
    const NormCols<T, V> cols{lane * V - m, a.tpr * V, a.D};
    const T* px = static_cast<const T*>(a.x) + (lane * V - m) + first * a.ldx;  // the row to copy next
    const T* pg = static_cast<const T*>(a.dy) + (lane * V - m) + first * a.lddy;
    const T *qx = px, *qg = pg;                                           // the row to work on
    T* pd = static_cast<T*>(a.dx) + (lane * V - m) + first * (int64_t)a.D;
    Vec<WT, V> w[NV];
    P dw[NV][L::N], db[NV][L::N];
    auto fetch = [&](int left, int slot) {  // left: rows from this one to the last
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (cols.any(i)) {
                    if constexpr (SHIFT) {
                        const int n = min(V, a.D - cols.at(i));
                        ringx.copy(slot, i, px + i * a.tpr * V, n);
                        ringg.copy(slot, i, pg + i * a.tpr * V, n);
                    } else {
                        ringx.copy(slot, i, px + i * a.tpr * V);
                        ringg.copy(slot, i, pg + i * a.tpr * V);
                    }
                }
        }
        px += stepx;
        pg += stepg;
        Ring::commit();
    };
    const float *pm = a.mean + first, *pr = a.rstd + first;
    float mean_next = first < R ? *pm : 0.0f, rstd_next = first < R ? *pr : 0.0f;
    int left = R - first;  // rows from the thread's current one to the last
#pragma unroll
    for (int j = 0; j < DEP; ++j) fetch(left - j * step, j);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (cols.any(i)) w[i] = cols.template weight<WT>(i, a.w);
#pragma unroll
        for (int k = 0; k < L::N; ++k) dw[i][k] = db[i][k] = pset<V>(0.0f);
    }
    const float inv = 1.0f / (float)a.D;
    int slot = 0;
    for (int rest = R - blockIdx.x * rpb; rest > 0;
         rest -= step, left -= step, qx += stepx, qg += stepg, pd += stepd) {
        const bool on = left > 0;
        const float rstd = rstd_next;
        const P minus = pset<V>(-mean_next), r2 = pset<V>(rstd);
        pm += step;
        pr += step;
        if (left > step) {
            mean_next = *pm;
            rstd_next = *pr;
        }
        P xc[NV][L::N], gw[NV][L::N];  // x - mean and dy w
        P s0 = pset<V>(0.0f), s1 = pset<V>(0.0f);
        Ring::wait();
        if (on) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (cols.any(i)) {
                    Vec<T, V> cx = ringx.get(slot, i, qx + i * a.tpr * V);
                    Vec<T, V> cg = ringg.get(slot, i, qg + i * a.tpr * V);
                    if (SHIFT) {  // dy = 0 where there is no column: nothing is added there
                        cols.clear(i, cx);
                        cols.clear(i, cg);
                    }
#pragma unroll
                    for (int k = 0; k < L::N; ++k) {
                        const P n = padd(pbits<T, V>(cx, k), minus), d = pbits<T, V>(cg, k);
                        xc[i][k] = n;
                        dw[i][k] = pfma(pmul(d, r2), n, dw[i][k]);
                        db[i][k] = padd(db[i][k], d);
                        const P g = pmul(d, pbits<WT, V>(w[i], k));
                        gw[i][k] = g;
                        s0 = padd(s0, g);
                        s1 = pfma(g, n, s1);
                    }
                }
            }
        }
        float s[2] = {psum(s0), psum(s1)};
        row_sum<2>(s, a.tpr, red);
        fetch(left - DEP * step, slot);  // behind the sums that used the slots' last rows
        slot = slot + 1 == DEP ? 0 : slot + 1;
        if (on) {
            // dx = rstd g + c1 n + c0 with n = (x - mean) rstd formed again: a factor for x - mean would be
            // rstd^3 s1 / D, and powers of rstd leave fp32 for rows of spread 1e13 or 1e-13
            const P c0 = pset<V>(-rstd * (s[0] * inv)), c1 = pset<V>(-rstd * (s[1] * inv * rstd));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                keep_packed(w[i]);  // not kept widened in twice the registers
                if (cols.any(i)) {
                    P o[L::N];
#pragma unroll
                    for (int k = 0; k < L::N; ++k) {
                        o[k] = pfma(gw[i][k], r2, pfma(pmul(xc[i][k], r2), c1, c0));
                    }
                    if constexpr (SHIFT) cols.store(i, pd + i * a.tpr * V, o);
                    else pstore<T, V>(pd + i * a.tpr * V, o);
                }
            }
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.D;
    auto each = [&](auto f) {  // f(column, dw, db) for this thread's columns
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < L::N; ++k) {
                float x[2], y[2];
                if constexpr (V == 1) {
                    x[0] = dw[i][k];
                    y[0] = db[i][k];
                } else {
                    up2(dw[i][k], x[0], x[1]);
                    up2(db[i][k], y[0], y[1]);
                }
#pragma unroll
                for (int h = 0; h < (V == 1 ? 1 : 2); ++h) {
                    const int c = cols.at(i) + 2 * k + h;
                    if (c >= 0 && c < a.D) f(c, x[h], y[h]);
                }
            }
    };
    if (rpb == 1) {
        each([&](int c, float x, float y) {
            part[c] = x;
            part[a.D + c] = y;
        });
        return;
    }
    // the rows of a block, joined one after the other (their order is fixed)
    float* acc = reinterpret_cast<float*>(norm_smem);
    __syncthreads();  // every thread is done with its ring
    for (int r = 0; r < rpb; ++r) {
        __syncthreads();
        if (sub == r)
            each([&](int c, float x, float y) {
                acc[c] = (r ? acc[c] : 0.0f) + x;
                acc[a.D + c] = (r ? acc[a.D + c] : 0.0f) + y;
            });
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

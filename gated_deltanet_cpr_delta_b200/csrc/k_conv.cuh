// k_conv.cuh -- the short causal convolution of a packed batch (sm_100a).
//
// Per sequence and channel c, with W = 2..4 taps and earlier inputs from the
// cached state (zeros without one):
//     pre[t] = bias + sum_{i<W} w[c][i] x[t - (W-1) + i],   y[t] = act(pre[t])
// with act = silu or the identity.  Its gradients, with g = dy act'(pre):
//     dx[t] = sum_j w[c][W-1-j] g[t+j],   dw[c][i] = sum_t g[t] x[t - (W-1) + i]
//
// Bound by memory: one read of x (and dy) and one write.  A thread keeps a
// rolling window of W rows of four channels in registers (as packed fp32 pairs) and
// walks a run of tokens, so that x is read once plus W-1 rows per run, which the
// neighbouring run brings into L2 anyway.  Runs are as long as one full wave of
// blocks allows.  Measured on a B200 (bf16, W = 4, silu): forward of 16384 x 6144
// 73 us, 5.5 TB/s, 85% of the copy rate, with two special-function instructions per element
// (48 us) next to it; gradients of 16384 x 2048 56 us + 4 us for the
// sums of dw, 3.6 TB/s; the step of 64 x 12288 3.9 us.  Rows that are not whole 8 bytes
// go in groups of 2 channels or singly: 8192 x 4097 39 us, gradients 105 us (x 4096: 27, 56).
#pragma once

#include "layer_common.cuh"

namespace gdn {

struct ConvArgs {
    Seqs s;
    const void* x;
    int64_t ldx;
    const void *w, *bias;
    const void* state_in;
    int32_t D;
    int silu, w_bf16;
    // forward
    void *y, *state_out;
    // backward
    const void* dy;
    int64_t lddy;
    const float* dstate_out;
    void* dx;
    float *dstate_in, *part;
    // grid: ncb channel blocks x (token tiles, then one state tile per sequence)
    int32_t ncb, cx;  // cx threads along the channels, 128 / cx runs of tokens per block
    int64_t ntiles;
    int32_t run;      // tokens per run
    int32_t* status;
};

// The taps and the window hold pairs of channels (or one channel, V = 1).
template <typename T, int W, int V>
struct ConvTaps {
    using P = typename Lanes<V>::type;
    static constexpr int N = Lanes<V>::N;
    P w[W][N], b[N];
    __device__ __forceinline__ void load(const ConvArgs& a, int64_t c)
    {
        float raw[V * W], rb[V];
        load_ws<V * W>(a.w, a.w_bf16, c * W, raw);
#pragma unroll
        for (int v = 0; v < V; ++v) rb[v] = 0.0f;
        if (a.bias != nullptr) load_ws<V>(a.bias, a.w_bf16, c, rb);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (V == 1) {
                b[n] = rb[0];
#pragma unroll
                for (int i = 0; i < W; ++i) w[i][n] = raw[i];
            } else {
                b[n] = pk2(rb[2 * n], rb[2 * n + 1]);
#pragma unroll
                for (int i = 0; i < W; ++i) w[i][n] = pk2(raw[2 * n * W + i], raw[(2 * n + 1) * W + i]);
            }
        }
    }
    __device__ __forceinline__ P pre(const P (&win)[W][N], int n) const
    {
        P p = b[n];
#pragma unroll
        for (int i = 0; i < W; ++i) p = pfma(w[i][n], win[i][n], p);
        return p;
    }
};

// f on every element of a pair
template <typename F>
__device__ __forceinline__ f2x peach(f2x a, F f)
{
    float x, y;
    up2(a, x, y);
    return pk2(f(x), f(y));
}
template <typename F>
__device__ __forceinline__ float peach(float a, F f) { return f(a); }

// The window before row t of sequence n: win[i] = x[t - (W-1) + i] for i < W-1.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_window(const ConvArgs& a, int n, int64_t lo, int64_t t, int64_t c,
                                            typename Lanes<V>::type (&win)[W][Lanes<V>::N])
{
    const T* x = static_cast<const T*>(a.x);
    const T* st = static_cast<const T*>(a.state_in);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int64_t r = t - (W - 1) + i;
        Vec<T, V> v;
        bool have = true;
        if (r >= lo) v = load_vec<T, V>(x + r * a.ldx + c);
        else if (st != nullptr) v = load_vec<T, V>(st + ((int64_t)n * (W - 1) + (W - 1) + (r - lo)) * a.D + c);
        else have = false;
#pragma unroll
        for (int k = 0; k < Lanes<V>::N; ++k) win[i][k] = have ? pget<T, V>(v, k) : pset<V>(0.0f);
    }
}

// A thread's own rows ahead, in a ring in shared memory that cp.async fills (4, 8 or 16
// bytes a row; 2-byte rows are loaded when they are needed).  In registers the rows ahead
// cost the occupancy that they were to spare: the gradients held 125 registers and 4
// blocks per SM with 8 rows of 2 channels ahead.
template <typename T, int V, int DEP>
struct ConvRing {
    static constexpr int B = V * sizeof(T);
    static constexpr bool ON = B >= 4;
    static constexpr size_t BYTES = ON ? (size_t)DEP * 128 * B : 0;  // per tensor
    unsigned char* base;
    __device__ __forceinline__ unsigned char* at(int slot) const { return base + (slot * 128 + threadIdx.x) * B; }
    __device__ __forceinline__ void copy(int slot, const T* src) const
    {
        if constexpr (ON) {
            const unsigned to = (unsigned)__cvta_generic_to_shared(at(slot));
            if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
            else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(B) : "memory");
        }
    }
    __device__ __forceinline__ Vec<T, V> get(int slot, const T* src) const
    {
        if constexpr (ON) return *reinterpret_cast<const Vec<T, V>*>(at(slot));
        else return load_vec<T, V>(src);
    }
    __device__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    __device__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEP - 1) : "memory"); }
};

constexpr int kConvAhead = 8;  // rows ahead

// state_out of one sequence: its last W-1 inputs, the old state's where it is shorter.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_tail(const ConvArgs& a, int n, int64_t c)
{
    const int64_t lo = a.s.lo(n), L = a.s.hi(n) - lo;
    const T* x = static_cast<const T*>(a.x);
    const T* st = static_cast<const T*>(a.state_in);
    T* out = static_cast<T*>(a.state_out) + (int64_t)n * (W - 1) * a.D + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int64_t p = L - (W - 1) + i;
        Vec<T, V> v;
        if (p >= 0) v = load_vec<T, V>(x + (lo + p) * a.ldx + c);
        else if (st != nullptr) v = load_vec<T, V>(st + ((int64_t)n * (W - 1) + (W - 1) + p) * a.D + c);
        else {
#pragma unroll
            for (int k = 0; k < V; ++k) v.v[k] = from_f<T>(0.0f);
        }
        *reinterpret_cast<Vec<T, V>*>(out + (int64_t)i * a.D) = v;
    }
}

// Where kConvAhead rows lie in one sequence (almost everywhere) there is no test per row.
template <typename T, int W, int V>
__global__ void __launch_bounds__(128, 7) k_conv_fwd(const ConvArgs a)
{
    constexpr int U = kConvAhead;
    extern __shared__ __align__(16) unsigned char conv_smem[];
    const ConvRing<T, V, U> ring{conv_smem};
    if (blockIdx.x == 0) check_seqs(a.s, a.status);
    const int64_t tile = blockIdx.x / a.ncb;
    const int cb = (int)(blockIdx.x - tile * a.ncb);
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx, ny = 128 / a.cx;
    const int64_t c = ((int64_t)cb * a.cx + tx) * V;
    if (c >= a.D) return;
    if (tile >= a.ntiles) {
        const int64_t n = (tile - a.ntiles) * ny + ty;
        if (n < a.s.N) conv_tail<T, W, V>(a, (int)n, c);
        return;
    }
    const int64_t t64 = (tile * ny + ty) * a.run;
    if (t64 >= a.s.T) return;
    int t = (int)t64;  // rows are below 2^31
    const int end = (int)min(t64 + a.run, a.s.T);
    int n = a.s.find(t);
    if (n < 0) {  // rows before the first sequence
        t = (int)min(a.s.lo(0), (int64_t)end);
        if (t >= end) return;
        n = a.s.find(t);
    }
    ConvTaps<T, W, V> taps;
    taps.load(a, c);
    const int64_t ldx = a.ldx, ldy = a.D;
    const T* x = static_cast<const T*>(a.x) + c + t * ldx;  // row t
    T* y = static_cast<T*>(a.y) + c + t * ldy;
    int hi = (int)a.s.hi(n);
    using P = typename Lanes<V>::type;
    constexpr int N = Lanes<V>::N;
    P win[W][N];
    conv_window<T, W, V>(a, n, a.s.lo(n), t, c, win);
    auto row = [&](const Vec<T, V>& r, T* out, bool store) {
        P o[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            win[W - 1][k] = pget<T, V>(r, k);
            o[k] = taps.pre(win, k);
            if (a.silu) o[k] = pmul(o[k], peach(o[k], sigmoid));
#pragma unroll
            for (int i = 0; i < W - 1; ++i) win[i][k] = win[i + 1][k];
        }
        if (store) pstore<T, V>(out, o);
    };
    const T* px = x;  // the row to copy next
    auto fetch = [&](int slot, bool in) {
        if (in) ring.copy(slot, px);
        px += ldx;
        ring.commit();
    };
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, t + u < end);
    for (; t < end; t += U) {
        if (!ring.ON && t + U <= min(hi, end)) {  // 2-byte rows: all loads before the first use
            Vec<T, V> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = load_vec<T, V>(x + u * ldx);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                row(raw[u], y, true);
                y += ldy;
            }
            x += U * ldx;
        } else if (t + U <= min(hi, end)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ring.wait();
                row(ring.get(u, x), y, true);
                fetch(u, t + U + u < end);  // behind the store that used the slot's last row
                x += ldx;
                y += ldy;
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < U && t + u < end; ++u) {
                if (t + u >= hi && n + 1 < a.s.N && t + u >= a.s.lo(n + 1)) {  // the next sequence's first token
                    n = a.s.find(t + u);
                    hi = (int)a.s.hi(n);
                    conv_window<T, W, V>(a, n, a.s.lo(n), t + u, c, win);
                }
                ring.wait();
                row(ring.get(u, x), y, t + u < hi);  // rows behind the last sequence stay
                fetch(u, t + U + u < end);
                x += ldx;
                y += ldy;
            }
        }
    }
}

// Gradients.  acc[i] is the unfinished dx of row t - (W-1) + i; after row t is
// added, acc[0] is finished.  At a sequence's end the W-1 open rows are
// finished too: they are the rows that the final state holds, in its order, so
// dstate_out[i] is added to acc[i].  A row before the sequence's start is a row of
// the initial state: its sum goes to dstate_in.  A run owns the rows [t0, t1)
// and reads on up to W-1 rows behind them; a state tile owns the rows before
// the start.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_bwd_run(const ConvArgs& a, int64_t t0, int64_t t1, int only_seq, int64_t c,
                                             const ConvTaps<T, W, V>& taps, typename Lanes<V>::type (&dw)[W][Lanes<V>::N],
                                             typename Lanes<V>::type (&db)[Lanes<V>::N], unsigned char* smem)
{
    const ConvRing<T, V, kConvAhead> ringx{smem}, ringg{smem + ConvRing<T, V, kConvAhead>::BYTES};
    using P = typename Lanes<V>::type;
    constexpr int N = Lanes<V>::N;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.dx);
    int64_t t = t0;
    int n = only_seq >= 0 ? only_seq : a.s.find(t);
    if (n < 0) {
        t = min(a.s.lo(0), t1);
        if (t >= t1) return;
        n = a.s.find(t);
    }
    while (true) {  // one sequence's part of the run per pass
        const int64_t lo = a.s.lo(n), hi = a.s.hi(n);
        // rows this pass reads, and the last row it may add to a row that it owns
        const int64_t stop = only_seq >= 0 ? min(hi, lo + (W - 1)) : min(hi, t1 + (W - 1));
        P win[W][N], acc[W][N];
        conv_window<T, W, V>(a, n, lo, t, c, win);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int k = 0; k < N; ++k) acc[i][k] = pset<V>(0.0f);
        auto emit = [&](int64_t r, const P (&v)[N]) {
            if (only_seq >= 0) {
                if (r < lo) pstore<float, V>(a.dstate_in + ((int64_t)n * (W - 1) + (W - 1) + (r - lo)) * a.D + c, v);
            } else if (r >= lo && r >= t0 && r < t1) {
                pstore<T, V>(dx + r * a.D + c, v);
            }
        };
        // One row.  `inner`: the row and the finished one are the run's own.
        auto row = [&](const Vec<T, V>& rx, const Vec<T, V>& rg, int64_t at, T* out, bool inner) {
            const bool own = inner || at < t1;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                win[W - 1][k] = pget<T, V>(rx, k);
                P g = pget<T, V>(rg, k);
                if (a.silu) g = pmul(g, peach(taps.pre(win, k), silu_grad));
                const P go = own ? g : pset<V>(0.0f);
                db[k] = padd(db[k], go);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    acc[i][k] = i < W - 1 ? pfma(taps.w[i][k], g, acc[i][k]) : pmul(taps.w[i][k], g);
                    dw[i][k] = pfma(go, win[i][k], dw[i][k]);
                }
            }
            if (inner) pstore<T, V>(out, acc[0]);
            else emit(at - (W - 1), acc[0]);
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    win[i][k] = win[i + 1][k];
                    acc[i][k] = acc[i + 1][k];
                }
        };
        constexpr int U = kConvAhead;
        const int64_t ldx = a.ldx, ldg = a.lddy;
        const T* px = x + t * ldx + c;  // row t
        const T* pg = dy + t * ldg + c;
        T* pd = dx + (t - (W - 1)) * (int64_t)a.D + c;  // the row finished at t
        const int64_t first = max(lo, t0) + (W - 1), last = only_seq >= 0 ? first : min(stop, t1);
        const T *cx = px, *cg = pg;  // the rows to copy next
        auto fetch = [&](int slot, bool in) {
            if (in) {
                ringx.copy(slot, cx);
                ringg.copy(slot, cg);
            }
            cx += ldx;
            cg += ldg;
            ringx.commit();
        };
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(u, t + u < stop);
        auto step = [&](int u, bool inner) {
            ringx.wait();
            row(ringx.get(u, px), ringg.get(u, pg), t + u, pd, inner);
            fetch(u, t + U + u < stop);  // behind the use of the slots' last rows
            px += ldx;
            pg += ldg;
            pd += a.D;
        };
        for (; t < stop; t += U) {
            if (!ringx.ON && t >= first && t + U <= last) {  // 2-byte rows: all loads before the first use
                Vec<T, V> rx[U], rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rx[u] = load_vec<T, V>(px + u * ldx);
                    rg[u] = load_vec<T, V>(pg + u * ldg);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) row(rx[u], rg[u], t + u, pd + u * (int64_t)a.D, true);
                px += U * ldx;
                pg += U * ldg;
                pd += U * (int64_t)a.D;
            } else if (t >= first && t + U <= last) {
#pragma unroll
                for (int u = 0; u < U; ++u) step(u, true);
            } else {
#pragma unroll 1
                for (int u = 0; u < U && t + u < stop; ++u) step(u, false);
            }
        }
        if (stop == hi) {  // the sequence's end: the open rows hi - (W-1) + i
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                if (a.dstate_out != nullptr) {
                    const Vec<float, V> v =
                        load_vec<float, V>(a.dstate_out + ((int64_t)n * (W - 1) + i) * a.D + c);
#pragma unroll
                    for (int k = 0; k < N; ++k) acc[i][k] = padd(acc[i][k], pget<float, V>(v, k));
                }
                emit(hi - (W - 1) + i, acc[i]);
            }
        }
        if (only_seq >= 0 || hi >= t1) return;
        // the next sequence of this run
        if (n + 1 >= a.s.N) return;
        t = max(hi, a.s.lo(n + 1));
        if (t >= t1) return;
        const int m = a.s.find(t);
        if (m <= n) return;
        n = m;
    }
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(128, 4) k_conv_bwd(const ConvArgs a)
{
    extern __shared__ __align__(16) unsigned char conv_smem[];
    unsigned char* smem = conv_smem;                  // two rings; then
    float* sh = reinterpret_cast<float*>(conv_smem);  // [(W + 1) * V][128]: joins the runs of a block
    if (blockIdx.x == 0) check_seqs(a.s, a.status);
    const int64_t tile = blockIdx.x / a.ncb;
    const int cb = (int)(blockIdx.x - tile * a.ncb);
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx, ny = 128 / a.cx;
    const int64_t c = ((int64_t)cb * a.cx + tx) * V;
    using P = typename Lanes<V>::type;
    constexpr int N = Lanes<V>::N;
    P dw[W][N], db[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        db[k] = pset<V>(0.0f);
#pragma unroll
        for (int i = 0; i < W; ++i) dw[i][k] = pset<V>(0.0f);
    }
    if (c < a.D) {
        ConvTaps<T, W, V> taps;
        taps.load(a, c);
        if (tile >= a.ntiles) {
            const int64_t n = (tile - a.ntiles) * ny + ty;
            // no rows are owned: only the state's gradient is written
            if (n < a.s.N) conv_bwd_run<T, W, V>(a, a.s.lo((int)n), a.s.lo((int)n), (int)n, c, taps, dw, db, smem);
        } else {
            const int64_t t0 = (tile * ny + ty) * a.run, t1 = min(t0 + a.run, a.s.T);
            if (t0 < t1) conv_bwd_run<T, W, V>(a, t0, t1, -1, c, taps, dw, db, smem);
        }
    }
    if (tile >= a.ntiles) return;
    __syncthreads();  // every thread is done with its rings
#pragma unroll
    for (int i = 0; i <= W; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const P v = i < W ? dw[i < W ? i : 0][k] : db[k];
            if constexpr (V == 1) {
                sh[i * 128 + threadIdx.x] = v;
            } else {
                float x, y;
                up2(v, x, y);
                sh[(i * V + 2 * k) * 128 + threadIdx.x] = x;
                sh[(i * V + 2 * k + 1) * 128 + threadIdx.x] = y;
            }
        }
    __syncthreads();
    if (ty == 0 && c < a.D) {
#pragma unroll
        for (int j = 0; j < (W + 1) * V; ++j) {
            float s = 0.0f;
            for (int r = 0; r < ny; ++r) s += sh[j * 128 + r * a.cx + tx];
            a.part[(tile * (W + 1) + j / V) * a.D + c + j % V] = s;
        }
    }
}

// [W + 1][D] column sums -> dweight [D][W] and dbias [D]
struct ConvGradMap {
    float *dw, *db;
    int32_t D, W;
    __device__ void operator()(int64_t m, float s) const
    {
        const int i = (int)(m / D);
        const int64_t c = m - (int64_t)i * D;
        if (i < W) dw[c * W + i] = s;
        else if (db != nullptr) db[c] = s;
    }
};

// One token per sequence: window = [state, x]; state_out = the window without its first row.
template <typename T, int W, int V>
__global__ void __launch_bounds__(128) k_conv_step(const T* __restrict__ x, int64_t ldx, const void* w,
                                                   const void* bias, const T* state, T* state_out, int64_t N,
                                                   int32_t D, int silu_on, int w_bf16, T* __restrict__ y)
{
    const int64_t per = D / V;
    const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (id >= N * per) return;
    const int64_t n = id / per, c = (id - n * per) * V;
    Vec<T, V> win[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) win[i] = load_vec<T, V>(state + (n * (W - 1) + i) * D + c);
    win[W - 1] = load_vec<T, V>(x + n * ldx + c);
    float o[V], taps[V * W];
    load_ws<V * W>(w, w_bf16, c * W, taps);
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = 0.0f;
    if (bias != nullptr) load_ws<V>(bias, w_bf16, c, o);
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int i = 0; i < W; ++i) o[k] = __fmaf_rn(taps[k * W + i], to_f<T>(win[i].v[k]), o[k]);
        if (silu_on) o[k] = silu(o[k]);
    }
    store_vec<T, V>(y + n * D + c, o);
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
        *reinterpret_cast<Vec<T, V>*>(state_out + (n * (W - 1) + i) * D + c) = win[i + 1];
}

}  // namespace gdn

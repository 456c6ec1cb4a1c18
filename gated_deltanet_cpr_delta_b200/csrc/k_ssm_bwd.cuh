// k_ssm_bwd.cuh -- gradients of the selective state space scan (sm_100a).
//
// With a_t = exp(delta A), u = delta x, y' = sum_s h_t C + D x, dy' = dy silu(z)
// and e the gradient for the state after the token (from the tokens behind it):
//     g_t = C_t dy'_t + e_{t+1}                 (dL/dh_t)
//     e_t = a_t g_t                             (dL/dh_{t-1} from t on)
//     dC_t = sum_c dy' h_t,   dB_t = sum_c g u  (over the channels of the group)
//     dx   = delta sum_s g B + D dy',   dD = sum_t dy' x,   dz = dy y' silu'(z)
//     dA   = sum_t delta g (a_t h_{t-1})
//     ddelta = sum_s g (a_t h_{t-1}) A + x sum_s g B,   ddt = ddelta softplus'(dt + bias)
//
// Time is cut into chunks of Lc tokens, so that few channels fill the GPU: k_ssm_rev finds
// each chunk's e from zero, k_ssm_bwd_pass carries it over the chunks, then k_ssm_bwd walks
// the chunks in parallel.  A chunk is walked in reverse in parts of 32 tokens, each
// from the state that the forward saved there.  A part runs forward once,
// leaving the state before every 4th token in shared memory; then the 4-token
// tiles run in reverse: a tile is recomputed from its state, its 4 decays and
// decayed states stay in registers, and the adjoint walks back over them.  A
// decay is made twice, not three times.
//
// A lane holds 4 states of 2 channels, which leaves room for the tile's 64 registers of
// decays and states.  dB and dC are sums over the
// channels: 8 values per lane, summed over the lanes that share the states and over
// the warps in shared memory, and over the channel blocks by k_ssm_dbc, in a fixed order.
//
// Bound by instructions and their latency: 30 per (token, channel, state) in k_ssm_bwd, at
// half of the issue slots with 12 warps per SM (168 registers, 72 KB).  Measured on a B200 for
// 2 x 4096 tokens x 2048 channels x 16 states (bf16): k_ssm_rev 107 us, k_ssm_bwd_pass
// 7 us, k_ssm_bwd 449 us, the sums 24 us; the exponentials (three per element) take
// 173 us of that.  The forward's form (time segments in lanes, each exponential made
// once, the channels in a loop) took 718 us in place of the three: as many instructions,
// and half the warps.  Rows that are not whole 16 bytes load element by element:
// 8192 tokens x 4096 channels 1190 us in all, x 4097 1620 us.  4 x 2048 x 2048: 584, 1198 and 3051 us at 16, 32
// and 64 states.
#pragma once

#include "k_ssm.cuh"

namespace gdn {

constexpr int kSsmThreads = 128;
constexpr int kSsmTile = 16;   // tokens that k_ssm_rev stages together

template <int S>
struct SsmRevCfg {
    static constexpr int LN = S / 4;              // lanes per channel
    static constexpr int CW = 4 * (32 / LN);      // channels per warp
    static constexpr int CB = CW * (kSsmThreads / 32);
};

// Sum over the LN lanes of a channel, of 4 values (one per channel of the
// lane): returns the sum of channel ssm_own<LN>(lane).
template <int LN>
__device__ __forceinline__ float sum_channels(float v0, float v1, float v2, float v3, int q)
{
    constexpr int H1 = LN / 2, H2 = LN / 4;
    const bool up = (q & H1) != 0;
    const float s0 = up ? v0 : v2, s1 = up ? v1 : v3;
    float k0 = up ? v2 : v0, k1 = up ? v3 : v1;
    k0 += __shfl_xor_sync(kFullMask, s0, H1);
    k1 += __shfl_xor_sync(kFullMask, s1, H1);
    const bool odd = (q & H2) != 0;
    const float s = odd ? k0 : k1;
    float k = odd ? k1 : k0;
    k += __shfl_xor_sync(kFullMask, s, H2);
#pragma unroll
    for (int o = H2 / 2; o > 0; o >>= 1) k += __shfl_xor_sync(kFullMask, k, o);
    return k;
}
template <int LN>
__device__ __forceinline__ int ssm_own(int q)
{
    return ((q & (LN / 2)) ? 2 : 0) + ((q & (LN / 4)) ? 1 : 0);
}

struct SsmBwdArgs {
    SsmArgs f;
    int64_t Lc;         // tokens per chunk (a multiple of kSsmTile and kSsmSave)
    float *ebuf, *dsum; // [slots][D][S] the adjoint that enters each chunk from behind, [slots][D] sums of delta
    const void* dy;
    int64_t lddy;
    const float* dstate_out;
    void *dx, *ddt, *dz;
    float* dstate_in;
    float *partA;       // [slots][D][S]
    float *partD;       // [slots][2][D]: dD, ddt_bias
    float *partBC;      // [channel blocks per group][T][G][2 S]
};

template <int S>
struct SsmBwdCfg {
    static constexpr int LN = S / 4;
    static constexpr int CW = 2 * (32 / LN);
    static constexpr int CB = CW * (kSsmThreads / 32);
    static constexpr int SLOT = S > 32 ? 8 * S : 256;  // floats per warp and 4-token tile: states, later dB and dC
    static constexpr int NT = kSsmSave / 4;
    static constexpr int NG = 32 / LN;                   // lanes that share their states
    static constexpr int PAIR = 2 * NG * 2 * S;          // floats per warp: dB and dC of 2 tokens and NG channel pairs
    static constexpr size_t SMEM =
        sizeof(float) * (3 * kSsmSave * CB + 2 * kSsmSave * S + 4 * NT * SLOT + 4 * PAIR);
};

// The adjoint of a chunk from zero, tokens in reverse: e = a (C dy' + e), and the chunk's
// sum of delta.  S / 4 lanes share 4 channels, 4 states each; the tokens are staged 16 at a time.
template <typename T, int S, int V>
__global__ void __launch_bounds__(kSsmThreads, 4) k_ssm_rev(const SsmBwdArgs b)
{
    using Cf = SsmRevCfg<S>;
    constexpr int LN = Cf::LN, CW = Cf::CW, CB = Cf::CB, TT = kSsmTile;
    constexpr int PER_ROW = CB / V;                            // vectors per token row
    constexpr int NVEC = (TT * PER_ROW + kSsmThreads - 1) / kSsmThreads;
    constexpr int RSTEP = kSsmThreads / PER_ROW;               // rows between a thread's vectors
    constexpr int NC = TT * S / kSsmThreads;                   // elements of C per thread and tile
    static_assert(kSsmThreads % PER_ROW == 0, "a thread's vectors share their columns");
    __shared__ __align__(16) float sd[TT][CB];                 // delta
    __shared__ __align__(16) float su[TT][CB];                 // dy'
    __shared__ __align__(16) float sC[TT][S];

    const SsmArgs& a = b.f;
    const int cpg = (a.Dg + CB - 1) / CB, nb = a.G * cpg;
    const int64_t slot = blockIdx.x / nb;
    const int cb = (int)(blockIdx.x - slot * nb), e = cb / cpg;
    const int cbase = e * a.Dg + (cb - e * cpg) * CB, cend = (e + 1) * a.Dg;  // this block's channels, below cend
    const int n = a.s.find_slot(slot, b.Lc);
    const int64_t lo = a.s.lo(n), L = a.s.hi(n) - lo, chunk = slot - a.s.first_slot(n, b.Lc);
    const int64_t nch = L > 0 ? (L + b.Lc - 1) / b.Lc : 1;
    if (chunk < 1 || chunk >= nch) return;                     // the first chunk's is made by its own walk
    const int64_t p0 = chunk * b.Lc, p1 = min(p0 + b.Lc, L);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LN - 1);
    const int col = warp * CW + (lane / LN) * 4;               // the lane's first column of the block
    f2x A2[4][2], h[4][2];                                     // A log2 e, and the adjoint
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = cbase + col + i;
        float4 av = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < cend) av = *reinterpret_cast<const float4*>(a.A + (int64_t)c * S + 4 * q);
        A2[i][0] = pk2(av.x * kLog2e, av.y * kLog2e);
        A2[i][1] = pk2(av.z * kLog2e, av.w * kLog2e);
        h[i][0] = h[i][1] = pk2(0.f, 0.f);
    }
    float dsum[4] = {0.f, 0.f, 0.f, 0.f};

    const int vc = (tid % PER_ROW) * V, vr = tid / PER_ROW;
    const bool vok = cbase + vc < cend;  // V divides Dg and cbase where V > 1
    const float* bias = a.dt_bias != nullptr && vok ? a.dt_bias + cbase + vc : nullptr;
    const T* x = static_cast<const T*>(b.dy) + cbase + vc;
    const T* dt = static_cast<const T*>(a.dt) + cbase + vc;
    const T* z = a.z != nullptr ? static_cast<const T*>(a.z) + cbase + vc : nullptr;
    const T* C = static_cast<const T*>(a.C) + e * S;

    Vec<T, V> rx[NVEC], rd[NVEC], rz[NVEC];
    T rc[NC];
    auto fetch = [&](int64_t p) {
#pragma unroll
        for (int i = 0; i < NVEC; ++i) {
            const int r = vr + i * RSTEP;
            if (vok && r < TT && p + r < p1) {
                const int64_t row = lo + p + r;
                rx[i] = load_vec<T, V>(x + row * b.lddy);
                rd[i] = load_vec<T, V>(dt + row * a.lddt);
                if (z != nullptr) rz[i] = load_vec<T, V>(z + row * a.ldz);
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int r = (i * kSsmThreads + tid) / S, s = (i * kSsmThreads + tid) % S;
            if (p + r < p1) rc[i] = C[(lo + p + r) * a.ldC + s];
        }
    };
    const f2x shift = pk2(kEx2Mean, kEx2Mean);
    const int64_t ntile = (p1 - p0 + TT - 1) / TT;
    fetch(p0 + (ntile - 1) * TT);
    for (int64_t it = ntile - 1; it >= 0; --it) {
        const int64_t p = p0 + it * TT;
        const int rows = (int)min((int64_t)TT, p1 - p);
#pragma unroll
        for (int i = 0; i < NVEC; ++i) {
            const int r = vr + i * RSTEP;
            if (r < TT) {
                const bool in = vok && r < rows;
                float vd[V], vu[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    vu[k] = in ? to_f<T>(rx[i].v[k]) : 0.0f;
                    if (z != nullptr && in) vu[k] *= silu(to_f<T>(rz[i].v[k]));
                    vd[k] = in ? ssm_delta(a, to_f<T>(rd[i].v[k]), bias != nullptr ? bias[k] : 0.0f) : 0.0f;
                }
                put_row<V>(&sd[r][vc], vd);
                put_row<V>(&su[r][vc], vu);
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) (&sC[0][0])[i * kSsmThreads + tid] = to_f<T>(rc[i]);
        __syncthreads();
        if (it > 0) fetch(p - TT);
#pragma unroll 2
        for (int t = rows - 1; t >= 0; --t) {
            const float4 d4 = *reinterpret_cast<const float4*>(&sd[t][col]);
            const float4 u4 = *reinterpret_cast<const float4*>(&su[t][col]);
            const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(&sC[t][4 * q]);
            const float d[4] = {d4.x, d4.y, d4.z, d4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2x d2 = pk2(d[i], d[i]), u2 = pk2(u[i], u[i]);
                float e0, e1, e2, e3;
                up2(ffma2(d2, A2[i][0], shift), e0, e1);
                up2(ffma2(d2, A2[i][1], shift), e2, e3);
                h[i][0] = fmul2(pk2(ex2(e0), ex2(e1)), ffma2(u2, c4.x, h[i][0]));
                h[i][1] = fmul2(pk2(ex2(e2), ex2(e3)), ffma2(u2, c4.y, h[i][1]));
                dsum[i] += d[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = cbase + col + i;
        float4 v;
        up2(h[i][0], v.x, v.y);
        up2(h[i][1], v.z, v.w);
        if (c < cend) {
            *reinterpret_cast<float4*>(b.ebuf + (slot * a.D + c) * S + 4 * q) = v;
            if (q == 0) b.dsum[slot * a.D + c] = dsum[i];
        }
    }
}

// Carries the adjoint back over the chunks: ebuf[chunk] becomes the gradient
// for the state after the chunk.
template <int S>
__global__ void __launch_bounds__(128) k_ssm_bwd_pass(const SsmBwdArgs b)
{
    const SsmArgs& a = b.f;
    const float* dstate_out = b.dstate_out;
    const int64_t per = (int64_t)a.D * (S / 4);
    const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (id >= per * a.s.N) return;
    const int n = (int)(id / per);
    const int64_t r = id - n * per;
    const int c = (int)(r / (S / 4)), s = (int)(r % (S / 4)) * 4;
    const int64_t L = a.s.hi(n) - a.s.lo(n), nch = (L + b.Lc - 1) / b.Lc;
    if (nch <= 1) return;
    const float4 av = *reinterpret_cast<const float4*>(a.A + (int64_t)c * S + s);
    const float A2[4] = {av.x * kLog2e, av.y * kLog2e, av.z * kLog2e, av.w * kLog2e};
    float e[4] = {0.f, 0.f, 0.f, 0.f};
    if (dstate_out != nullptr) {
        const float4 v = *reinterpret_cast<const float4*>(dstate_out + ((int64_t)n * a.D + c) * S + s);
        e[0] = v.x, e[1] = v.y, e[2] = v.z, e[3] = v.w;
    }
    // four chunks' parts are loaded together: the chain alone would wait for each
    constexpr int U = 4;
    float4* base = reinterpret_cast<float4*>(b.ebuf + (a.s.first_slot(n, b.Lc) * a.D + c) * S + s);
    const float* ds = b.dsum + a.s.first_slot(n, b.Lc) * a.D + c;
    const int64_t per_chunk = (int64_t)a.D * S / 4;
    for (int64_t k = nch - 1; k >= 0; k -= U) {
        float4 v[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            d[u] = 0.0f;
            if (k - u > 0) {  // the first chunk's part is made by its own walk
                v[u] = base[(k - u) * per_chunk];
                d[u] = ds[(k - u) * a.D];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k - u < 0) break;
            base[(k - u) * per_chunk] = make_float4(e[0], e[1], e[2], e[3]);
            e[0] = __fmaf_rn(ex2(d[u] * A2[0]), e[0], v[u].x);
            e[1] = __fmaf_rn(ex2(d[u] * A2[1]), e[1], v[u].y);
            e[2] = __fmaf_rn(ex2(d[u] * A2[2]), e[2], v[u].z);
            e[3] = __fmaf_rn(ex2(d[u] * A2[3]), e[3], v[u].w);
        }
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <typename T, int S, int V, bool GATE>
__global__ void __launch_bounds__(kSsmThreads, 3) k_ssm_bwd(const SsmBwdArgs b)
{
    using Cf = SsmBwdCfg<S>;
    constexpr int LN = Cf::LN, CW = Cf::CW, CB = Cf::CB, P = kSsmSave, NT = Cf::NT, NG = Cf::NG;
    constexpr int PER_ROW = CB / V;
    constexpr int RSTEP = kSsmThreads / PER_ROW;
    static_assert(kSsmThreads % PER_ROW == 0, "a thread's vectors share their columns");
    extern __shared__ __align__(16) float smem[];
    float* sd = smem;              // [P][CB] delta, then sum_s h C
    float* sx = sd + P * CB;       // x, then ddelta
    float* sg = sx + P * CB;       // dy', then dx
    float* sB = sg + P * CB;       // [P][S]
    float* sC = sB + P * S;
    float* sh = sC + P * S;        // [warps][NT][SLOT]
    float* sp = sh + 4 * NT * Cf::SLOT;  // [warps][PAIR]

    const SsmArgs& a = b.f;
    if (blockIdx.x == 0) check_seqs(a.s, a.status);
    const int nb = a.G * a.cpg;
    const int64_t slot = blockIdx.x / nb;
    const int cb = (int)(blockIdx.x - slot * nb), e = cb / a.cpg, cbg = cb - e * a.cpg;
    const int cbase = e * a.Dg + cbg * CB, cend = (e + 1) * a.Dg;
    const int n = a.s.find_slot(slot, b.Lc);
    const int64_t lo = a.s.lo(n), L = a.s.hi(n) - lo, chunk = slot - a.s.first_slot(n, b.Lc);
    const int64_t nch = L > 0 ? (L + b.Lc - 1) / b.Lc : 1;
    const bool idle = chunk < 0 || chunk >= nch;
    const int64_t p0 = idle ? 0 : chunk * b.Lc, p1 = idle ? 0 : min(p0 + b.Lc, L);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LN - 1);
    const int col = warp * CW + (lane / LN) * 2;
    float* tiles = sh + warp * NT * Cf::SLOT;
    float* pair = sp + warp * Cf::PAIR;
    const int grp = lane / LN;
    f2x A2[2][2], ev[2][2], dA[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = cbase + col + i;
        float4 av = make_float4(0.f, 0.f, 0.f, 0.f), w = av;
        if (c < cend && !idle) {
            av = *reinterpret_cast<const float4*>(a.A + (int64_t)c * S + 4 * q);
            const float* src = nullptr;
            if (nch > 1) src = b.ebuf + (slot * a.D + c) * S;
            else if (b.dstate_out != nullptr) src = b.dstate_out + ((int64_t)n * a.D + c) * S;
            if (src != nullptr) w = *reinterpret_cast<const float4*>(src + 4 * q);
        }
        A2[i][0] = pk2(av.x * kLog2e, av.y * kLog2e);
        A2[i][1] = pk2(av.z * kLog2e, av.w * kLog2e);
        ev[i][0] = pk2(w.x, w.y);
        ev[i][1] = pk2(w.z, w.w);
        dA[i][0] = dA[i][1] = pk2(0.f, 0.f);
    }
    const int own = ssm_own<LN>(q), oi = own & 1;  // 0, 1: ddelta of channel oi; 2, 3: dx of channel oi
    const bool owner = LN == 4 || (q & (LN / 4 - 1)) == 0;
    const int oc = cbase + col + oi;
    const float Do = a.Dp != nullptr && oc < cend ? a.Dp[oc] : 0.0f;
    float dD = 0.0f;

    const int vc = (tid % PER_ROW) * V, vr = tid / PER_ROW;
    const bool vok = cbase + vc < cend;
    __shared__ __align__(16) float sbias[CB], sD[CB];
    if (tid < CB) {
        const bool ok = cbase + tid < cend;
        sbias[tid] = ok && a.dt_bias != nullptr ? a.dt_bias[cbase + tid] : 0.0f;
        sD[tid] = ok && a.Dp != nullptr ? a.Dp[cbase + tid] : 0.0f;
    }
    __syncthreads();
    __shared__ __align__(16) float sdb[kSsmThreads * V];  // each thread's sums of ddt
    float* dbias = sdb + tid * V;
#pragma unroll
    for (int k = 0; k < V; ++k) dbias[k] = 0.0f;
    const T* x = static_cast<const T*>(a.x) + cbase + vc;
    const T* dt = static_cast<const T*>(a.dt) + cbase + vc;
    const T* dy = static_cast<const T*>(b.dy) + cbase + vc;
    const T* z = GATE ? static_cast<const T*>(a.z) + cbase + vc : nullptr;
    const T* B = static_cast<const T*>(a.B) + e * S;
    const T* C = static_cast<const T*>(a.C) + e * S;

    // one decay step of the lane's 8 state elements
    auto decay = [&](const float2 d, f2x (&o)[2][2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f2x d2 = pk2(i ? d.y : d.x, i ? d.y : d.x);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float e0, e1;
                up2(ffma2(d2, A2[i][k], pk2(kEx2Mean, kEx2Mean)), e0, e1);
                o[i][k] = pk2(ex2(e0), ex2(e1));
            }
        }
    };
    auto bcast = [](float v) { return pk2(v, v); };

    for (int64_t p = p0 + (p1 > p0 ? (p1 - p0 - 1) / P * P : -1); p >= p0; p -= P) {
        const int rows = (int)min((int64_t)P, p1 - p);
        if (p > p0) {  // the part before this one, on its way to L2
            for (int r = vr; r < P; r += RSTEP) {
                if (vok) {
                    const int64_t row = lo + p - P + r;
                    prefetch_l2(x + row * a.ldx);
                    prefetch_l2(dt + row * a.lddt);
                    prefetch_l2(dy + row * b.lddy);
                    if (GATE) prefetch_l2(z + row * a.ldz);
                }
            }
        }
        for (int r = vr; r < P; r += RSTEP) {
            const bool in = vok && r < rows;
            Vec<T, V> wx, wd, wg, wz;
            if (in) {
                const int64_t row = lo + p + r;
                wx = load_vec<T, V>(x + row * a.ldx);
                wd = load_vec<T, V>(dt + row * a.lddt);
                wg = load_vec<T, V>(dy + row * b.lddy);
                if (GATE) wz = load_vec<T, V>(z + row * a.ldz);
            }
            float vb[V], vd[V], vx[V], vg[V];
            get_row<V>(sbias + vc, vb);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                vd[k] = in ? ssm_delta(a, to_f<T>(wd.v[k]), vb[k]) : 0.0f;
                vx[k] = in ? to_f<T>(wx.v[k]) : 0.0f;
                vg[k] = in ? to_f<T>(wg.v[k]) * (GATE ? silu(to_f<T>(wz.v[k])) : 1.0f) : 0.0f;
            }
            put_row<V>(sd + r * CB + vc, vd);
            put_row<V>(sx + r * CB + vc, vx);
            put_row<V>(sg + r * CB + vc, vg);
        }
        for (int i = tid; i < P * S; i += kSsmThreads) {
            const int r = i / S, s = i % S;
            sB[i] = r < rows ? to_f<T>(B[(lo + p + r) * a.ldB + s]) : 0.0f;
            sC[i] = r < rows ? to_f<T>(C[(lo + p + r) * a.ldC + s]) : 0.0f;
        }
        f2x h[2][2];
        {
            const int64_t at = a.s.first_slot(n, kSsmSave) + p / kSsmSave;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = cbase + col + i;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < cend) v = *reinterpret_cast<const float4*>(a.saved + (at * a.D + c) * S + 4 * q);
                h[i][0] = pk2(v.x, v.y);
                h[i][1] = pk2(v.z, v.w);
            }
        }
        __syncthreads();
        // forward over the part: the state before every 4th token
        const int last = (rows - 1) / 4;
        for (int k = 0; k <= last; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<ulonglong2*>(tiles + k * Cf::SLOT + i * 128 + lane * 4) =
                    make_ulonglong2(h[i][0], h[i][1]);
            if (k == last) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * k + j;
                const float2 d = *reinterpret_cast<const float2*>(sd + t * CB + col);
                const float2 xv = *reinterpret_cast<const float2*>(sx + t * CB + col);
                const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(sB + t * S + 4 * q);
                f2x am[2][2];
                decay(d, am);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const f2x u2 = bcast(i ? d.y * xv.y : d.x * xv.x);
                    h[i][0] = ffma2(am[i][0], h[i][0], fmul2(u2, b4.x));
                    h[i][1] = ffma2(am[i][1], h[i][1], fmul2(u2, b4.y));
                }
            }
        }
        for (int k = last; k >= 0; --k) {
            f2x am[4][2][2], qm[4][2][2];
            float yk[4];  // sum_s h C of channel (q & LN / 2) != 0
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(tiles + k * Cf::SLOT + i * 128 + lane * 4);
                h[i][0] = v.x;
                h[i][1] = v.y;
            }
            __syncwarp();  // the tile's slot is rewritten below
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * k + j;  // rows behind `rows` hold delta = x = dy' = 0 and B = C = 0
                const float2 d = *reinterpret_cast<const float2*>(sd + t * CB + col);
                const float2 xv = *reinterpret_cast<const float2*>(sx + t * CB + col);
                const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(sB + t * S + 4 * q);
                decay(d, am[j]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const f2x u2 = bcast(i ? d.y * xv.y : d.x * xv.x);
                    qm[j][i][0] = fmul2(am[j][i][0], h[i][0]);
                    qm[j][i][1] = fmul2(am[j][i][1], h[i][1]);
                    h[i][0] = ffma2(u2, b4.x, qm[j][i][0]);
                    h[i][1] = ffma2(u2, b4.y, qm[j][i][1]);
                }
                if (GATE) {
                    const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(sC + t * S + 4 * q);
                    float o[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float ya, yb;
                        up2(ffma2(h[i][1], c4.y, fmul2(h[i][0], c4.x)), ya, yb);
                        o[i] = ya + yb;
                    }
                    const bool up = (q & (LN / 2)) != 0;
                    float s = (up ? o[1] : o[0]) + __shfl_xor_sync(kFullMask, up ? o[0] : o[1], LN / 2);
#pragma unroll
                    for (int w = LN / 4; w > 0; w >>= 1) s += __shfl_xor_sync(kFullMask, s, w);
                    yk[j] = s;
                }
            }
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const int t = 4 * k + j;
                const float2 d = *reinterpret_cast<const float2*>(sd + t * CB + col);
                const float2 xv = *reinterpret_cast<const float2*>(sx + t * CB + col);
                const float2 gv = *reinterpret_cast<const float2*>(sg + t * CB + col);
                const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(sB + t * S + 4 * q);
                const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(sC + t * S + 4 * q);
                const f2x bb[2] = {b4.x, b4.y}, cc[2] = {c4.x, c4.y};
                f2x dB[2], dC[2];
                float gB[2], dd[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float di = i ? d.y : d.x, xi = i ? xv.y : xv.x, gi = i ? gv.y : gv.x;
                    const f2x d2 = bcast(di), u2 = bcast(di * xi), g2 = bcast(gi);
                    f2x sgb = 0, sga = 0;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const f2x g = ffma2(cc[m], g2, ev[i][m]);
                        const f2x gq = fmul2(g, qm[j][i][m]);
                        const f2x ht = ffma2(u2, bb[m], qm[j][i][m]);
                        dA[i][m] = ffma2(d2, gq, dA[i][m]);
                        ev[i][m] = fmul2(am[j][i][m], g);
                        if (m == 0) {
                            sgb = fmul2(g, bb[m]);
                            sga = fmul2(gq, A2[i][m]);
                        } else {
                            sgb = ffma2(g, bb[m], sgb);
                            sga = ffma2(gq, A2[i][m], sga);
                        }
                        if (i == 0) {
                            dB[m] = fmul2(g, u2);
                            dC[m] = fmul2(ht, g2);
                        } else {
                            dB[m] = ffma2(g, u2, dB[m]);
                            dC[m] = ffma2(ht, g2, dC[m]);
                        }
                    }
                    float r0, r1;
                    up2(sgb, r0, r1);
                    gB[i] = r0 + r1;
                    up2(sga, r0, r1);
                    dd[i] = __fmaf_rn(xi, gB[i], (r0 + r1) * 0.6931471805599453f);
                }
                const float s = sum_channels<LN>(dd[0], dd[1], gB[0], gB[1], q);
                // this token's rows have been read by every lane of the warp (the shuffles order it)
                if (own >= 2) {
                    const float gi = oi ? gv.y : gv.x, xi = oi ? xv.y : xv.x, di = oi ? d.y : d.x;
                    dD = __fmaf_rn(gi, xi, dD);
                    if (owner) sg[t * CB + col + oi] = __fmaf_rn(di, s, Do * gi);
                } else if (owner) {
                    sx[t * CB + col + oi] = s;
                }
                if (GATE && (q & (LN / 2 - 1)) == 0) sd[t * CB + col + ((q & (LN / 2)) != 0 ? 1 : 0)] = yk[j];
                // dB and dC of this token: [channel pair][dB, dC][S], the halves of odd pairs swapped
                // (a quarter of the warp then writes to all banks); two tokens at a time are
                // summed over the channel pairs.  Halving by shuffles took 28 instructions
                // per token, this takes 12.
                float* w = pair + ((j & 1) * NG + grp) * 2 * S + 4 * q;
                *reinterpret_cast<ulonglong2*>(w + (grp & 1) * S) = make_ulonglong2(dB[0], dB[1]);
                *reinterpret_cast<ulonglong2*>(w + (~grp & 1) * S) = make_ulonglong2(dC[0], dC[1]);
                if ((j & 1) == 0) {
                    __syncwarp();
                    constexpr int OPL = S / 8;  // values per lane: 16 lanes to a token
                    const int tok = lane >> 4, at = (lane & 15) * OPL;
                    const float* r = pair + tok * NG * 2 * S;
                    f2x sum[OPL / 2];
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int k = 0; k < OPL / 2; ++k) {
                            const f2x x = *reinterpret_cast<const f2x*>(r + g * 2 * S + ((at + 2 * k) ^ ((g & 1) * S)));
                            sum[k] = g == 0 ? x : fadd2(sum[k], x);
                        }
                    float* o = tiles + k * Cf::SLOT + (j + tok) * 2 * S + at;
#pragma unroll
                    for (int k = 0; k < OPL / 2; ++k) *reinterpret_cast<f2x*>(o + 2 * k) = sum[k];
                    __syncwarp();
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < rows * 2 * S; i += kSsmThreads) {
            const int r = i / (2 * S), s = i % (2 * S);
            const float* t = sh + (r / 4) * Cf::SLOT + (r % 4) * 2 * S + s;
            float v = t[0];
#pragma unroll
            for (int w = 1; w < kSsmThreads / 32; ++w) v += t[w * NT * Cf::SLOT];
            b.partBC[(((int64_t)cbg * a.s.T + lo + p + r) * a.G + e) * 2 * S + s] = v;
        }
        for (int r = vr; r < rows; r += RSTEP) {
            if (!vok) break;
            const int64_t row = lo + p + r;
            float o[V], od[V], vb[V], sum[V];
            get_row<V>(dbias, sum);
            const Vec<T, V> wd = load_vec<T, V>(dt + row * a.lddt);
            get_row<V>(sg + r * CB + vc, o);
            get_row<V>(sx + r * CB + vc, od);
            get_row<V>(sbias + vc, vb);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (a.softplus) od[k] *= sigmoid(to_f<T>(wd.v[k]) + vb[k]);
                sum[k] += od[k];
            }
            put_row<V>(dbias, sum);
            store_vec<T, V>(static_cast<T*>(b.dx) + row * a.D + cbase + vc, o);
            store_vec<T, V>(static_cast<T*>(b.ddt) + row * a.D + cbase + vc, od);
            if (GATE) {
                const Vec<T, V> wx = load_vec<T, V>(x + row * a.ldx), wz = load_vec<T, V>(z + row * a.ldz);
                const Vec<T, V> wg = load_vec<T, V>(dy + row * b.lddy);
                get_row<V>(sd + r * CB + vc, o);
                get_row<V>(sD + vc, vb);
#pragma unroll
                for (int k = 0; k < V; ++k)
                    o[k] = to_f<T>(wg.v[k]) * silu_grad(to_f<T>(wz.v[k])) * __fmaf_rn(vb[k], to_f<T>(wx.v[k]), o[k]);
                store_vec<T, V>(static_cast<T*>(b.dz) + row * a.D + cbase + vc, o);
            }
        }
        __syncthreads();
    }
    // the gradient for the initial state, and this chunk's parts of the parameters' gradients
    float* ds = b.dstate_in + (int64_t)n * a.D * S;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = cbase + col + i;
        float4 v;
        if (c < cend) {
            up2(dA[i][0], v.x, v.y);
            up2(dA[i][1], v.z, v.w);
            *reinterpret_cast<float4*>(b.partA + (slot * a.D + c) * S + 4 * q) = v;
            if (!idle && chunk == 0) {
                up2(ev[i][0], v.x, v.y);
                up2(ev[i][1], v.z, v.w);
                *reinterpret_cast<float4*>(ds + (int64_t)c * S + 4 * q) = v;
            }
        }
    }
    if (own >= 2 && owner && oc < cend) b.partD[slot * 2 * a.D + oc] = dD;
    float* red = sd;  // [RSTEP][CB]
    static_assert(RSTEP * CB <= 3 * P * CB, "the token rows hold it");
#pragma unroll
    for (int k = 0; k < V; ++k) red[vr * CB + vc + k] = dbias[k];
    __syncthreads();
    if (tid < CB && cbase + tid < cend) {
        float s = 0.0f;
        for (int r = 0; r < RSTEP; ++r) s += red[r * CB + tid];
        b.partD[slot * 2 * a.D + a.D + cbase + tid] = s;
    }
}

// dB and dC [T][G][S] from the channel blocks' parts; rows outside every
// sequence are left as they are.
template <typename T, int S>
__global__ void __launch_bounds__(256) k_ssm_dbc(const Seqs s, const float* __restrict__ part, int32_t G, int32_t cpg,
                                                 T* __restrict__ dB, T* __restrict__ dC)
{
    const int64_t per = (int64_t)G * 2 * S, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= s.T * per) return;
    const int64_t row = id / per, i = id - row * per;
    const int n = s.find(row);
    if (n < 0 || row >= s.hi(n)) return;
    float v = 0.0f;
    for (int k = 0; k < cpg; ++k) v += part[(int64_t)k * s.T * per + id];
    const int g = (int)(i / (2 * S)), st = (int)(i % (2 * S));
    T* out = st < S ? dB : dC;
    out[(row * G + g) * S + (st < S ? st : st - S)] = from_f<T>(v);
}

struct PlainMap {
    float* out;
    __device__ void operator()(int64_t m, float s) const { out[m] = s; }
};

// [2][D] -> dD, ddt_bias (either may be unwanted)
struct SsmGradMap {
    float *dD, *dbias;
    int32_t D;
    __device__ void operator()(int64_t m, float s) const
    {
        if (m < D) {
            if (dD != nullptr) dD[m] = s;
        } else if (dbias != nullptr) {
            dbias[m - D] = s;
        }
    }
};

}  // namespace gdn

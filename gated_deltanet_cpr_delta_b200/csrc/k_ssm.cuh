// k_ssm.cuh -- the selective state space scan of a packed batch (sm_100a).
//
// Per channel c with group e(c), S states per channel, state h fp32:
//     delta = softplus(dt + dt_bias)  (or dt + dt_bias)
//     h_t[s] = exp(delta A[c][s]) h_{t-1}[s] + delta x B_t[e][s]
//     y_t    = (sum_s h_t[s] C_t[e][s] + D[c] x) silu(z_t)
//
// Bound by the exponentials: one per (token, channel, state), and an SM makes
// 16 a cycle against 128 fused multiply-adds, of which a state takes 4.  The
// decay is 2^(delta A log2 e), with A log2 e formed once per block.
//
// k_ssm_fwd serves prompts and training, k_ssm_step single tokens (bound by its state, read and
// written once: 64 x 4096 x 16 in 8.9 us, 4.0 TB/s).  Measured on a B200 for 4 x 4096
// tokens x 2048 channels x 16 states (bf16): 345 us, where the exponentials alone
// take 115 us and the bytes 42 us.  It issues 13 instructions per (token, channel,
// state) at 56% of the issue slots: 8 in the loop over the states, the rest for the
// step width, the gate, the staging and the joining of the segments.  Before it: two passes
// over chunks of time, every exponential made twice, 1022 us; this form with two
// channels per lane (168 registers, 12 warps per SM) 450 us.  Rows that are not whole 16
// bytes are staged element by element: 8192 tokens x 4096 channels 390 us, x 4097 517 us.
// 4 x 2048 tokens x 2048 channels: 175, 353 and 729 us at 16, 32 and 64 states.  A block walks its
// sequence alone: one of 32768 tokens takes 780 us at 64 channels as at 1024.
#pragma once

#include "layer_common.cuh"

namespace gdn {

constexpr int kSsmSave = 32;   // saved states: one every 32 tokens of a sequence (GDN_SSM_CHUNK)

struct SsmArgs {
    Seqs s;
    const void *x, *dt, *z, *B, *C;
    int64_t ldx, lddt, ldz, ldB, ldC;
    const float *A, *Dp, *dt_bias;
    int32_t D, G, Dg;   // channels, groups, channels per group
    int32_t cpg;        // channel blocks per group
    int softplus;
    int bc16;           // rows of B and C in 16-byte accesses
    const float* state_in;
    void* y;
    float *state_out, *saved;
    int32_t* status;
};

__device__ __forceinline__ float ssm_delta(const SsmArgs& a, float dt, float bias)
{
    const float v = dt + bias;
    return a.softplus ? softplus(v) : v;
}

// ------------------------------------------------------------------ forward
// One warp walks a sequence for 32 / SEG channels, tile by tile.  Its lanes
// are SEG time segments x 32 / SEG channels; a segment is 8 tokens, so a tile is
// 8 SEG tokens, and a lane keeps delta, delta x and y of its 8 tokens in registers.
// For each pair of states the lane makes its 8 decays once, runs its tokens
// from zero (the first segment from the carried state), the segments are joined by a
// warp scan of (product of decays, end state), and the lane runs its tokens
// again from its true state, with the decays it kept.  So every exponential is
// made once, sequences of few channels still fill the GPU, and y needs no sum
// over lanes.
template <typename T, int S, int SEG>
struct SsmFwdCfg {
    static constexpr int K = 8;                        // tokens per segment
    static constexpr int TT = K * SEG;                 // tokens per tile
    static constexpr int CL = 32 / SEG;                // channels per warp
    static constexpr int NW = 4;                       // warps per block
    static constexpr int CB = CL * NW;                 // channels per block
    static constexpr int THREADS = 32 * NW;
    // Token rows in shared memory: CB elements; 16 bytes of padding per segment
    // put the segments of a warp's access into different banks.
    static constexpr int SEGROW = K * CB + 16 / (int)sizeof(T);
    static constexpr int TOK = SEG * SEGROW;           // elements of a staged token tensor
    static constexpr int PS = SEG * (K + 2);           // float2 per state pair of a B or C plane
    static constexpr size_t BYTES = sizeof(T) * (2 * 3 * TOK + 2 * TT * S) + sizeof(float2) * 2 * (S / 2) * PS +
                                    sizeof(float) * 2 * S * CB;
};

// 16 bytes past L1, or 4 bytes (rows that are not whole 16-byte vectors)
template <int BYTES>
__device__ __forceinline__ void ssm_cp_async(void* smem, const void* gmem)
{
    const unsigned to = (unsigned)__cvta_generic_to_shared(smem);
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(gmem) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(gmem), "n"(BYTES) : "memory");
}

template <typename T, int S, int V, int SEG>
__global__ void __launch_bounds__(SsmFwdCfg<T, S, SEG>::THREADS, 4) k_ssm_fwd(const SsmArgs a)
{
    using Cf = SsmFwdCfg<T, S, SEG>;
    constexpr int K = Cf::K, TT = Cf::TT, CL = Cf::CL, CB = Cf::CB, NT = Cf::THREADS, NP = S / 2;
    extern __shared__ __align__(16) unsigned char ssm_smem[];
    T* raw = reinterpret_cast<T*>(ssm_smem);           // [2 stages][x, dt, z][TOK]
    T* rawB = raw + 2 * 3 * Cf::TOK;                   // [B, C][TT][S]
    float2* sB = reinterpret_cast<float2*>(rawB + 2 * TT * S);      // [NP][PS]
    float2* sC = sB + NP * Cf::PS;
    float2* sA = sC + NP * Cf::PS;                     // [NP][CB]: A log2 e
    float2* sH = sA + NP * CB;                         // [NP][CB]: the carried states

    if (blockIdx.x == 0) check_seqs(a.s, a.status);
    const int nb = a.G * a.cpg;
    const int n = blockIdx.x / nb, cb = blockIdx.x - n * nb, e = cb / a.cpg;
    const int cbase = e * a.Dg + (cb - e * a.cpg) * CB, cend = (e + 1) * a.Dg;
    const int64_t lo = a.s.lo(n), L = a.s.hi(n) - lo;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = lane / CL, ch = warp * CL + lane % CL;          // the lane's channel in the block
    const int ch0 = cbase + ch;
    const bool on = ch0 < cend;

    // parameters and initial states of the block's channels
    for (int i = tid; i < CB * S; i += NT) {
        const int c = i / S, st = i % S;
        const bool ok = cbase + c < cend;
        const int at = ((st / 2) * CB + c) * 2 + (st & 1);
        reinterpret_cast<float*>(sA)[at] = ok ? a.A[(int64_t)(cbase + c) * S + st] * kLog2e : 0.0f;
        reinterpret_cast<float*>(sH)[at] =
            ok && a.state_in != nullptr ? a.state_in[((int64_t)n * a.D + cbase + c) * S + st] : 0.0f;
    }
    const float bias = on && a.dt_bias != nullptr ? a.dt_bias[ch0] : 0.0f;
    const float Dv = on && a.Dp != nullptr ? a.Dp[ch0] : 0.0f;
    const T* B = static_cast<const T*>(a.B) + e * S;
    const T* C = static_cast<const T*>(a.C) + e * S;

    // a row's offset, from 32-bit factors (rows and strides are below 2^31)
    auto at = [](int row, int64_t ld) { return (int64_t)row * (int)ld; };
    auto stage = [&](int64_t p, int buf) {
        T* dst = raw + buf * 3 * Cf::TOK;
        const int rows = (int)min((int64_t)TT, L - p);
        if constexpr (V * sizeof(T) >= 4) {
            for (int i = tid; i < TT * (CB / V); i += NT) {
                const int t = i / (CB / V), v = (i % (CB / V)) * V;
                if (t < rows && cbase + v < cend) {
                    const int row = (int)(lo + p) + t;
                    T* d = dst + (t / K) * Cf::SEGROW + (t % K) * CB + v;
                    ssm_cp_async<V * sizeof(T)>(d, static_cast<const T*>(a.x) + at(row, a.ldx) + cbase + v);
                    ssm_cp_async<V * sizeof(T)>(d + Cf::TOK, static_cast<const T*>(a.dt) + at(row, a.lddt) + cbase + v);
                    if (a.z != nullptr)
                        ssm_cp_async<V * sizeof(T)>(d + 2 * Cf::TOK,
                                                    static_cast<const T*>(a.z) + at(row, a.ldz) + cbase + v);
                }
            }
        } else {  // 2 bytes: all loads before the first store
            constexpr int E = TT * CB / NT;
            T rx[E], rd[E], rz[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int t = (i * NT + tid) / CB, v = (i * NT + tid) % CB;
                if (t < rows && cbase + v < cend) {
                    const int row = (int)(lo + p) + t;
                    rx[i] = static_cast<const T*>(a.x)[at(row, a.ldx) + cbase + v];
                    rd[i] = static_cast<const T*>(a.dt)[at(row, a.lddt) + cbase + v];
                    if (a.z != nullptr) rz[i] = static_cast<const T*>(a.z)[at(row, a.ldz) + cbase + v];
                }
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int t = (i * NT + tid) / CB, v = (i * NT + tid) % CB;
                if (t < rows && cbase + v < cend) {
                    T* d = dst + (t / K) * Cf::SEGROW + (t % K) * CB + v;
                    d[0] = rx[i];
                    d[Cf::TOK] = rd[i];
                    if (a.z != nullptr) d[2 * Cf::TOK] = rz[i];
                }
            }
        }
    };
    constexpr int VB = 16 / (int)sizeof(T);            // states per 16-byte access
    auto stage_bc = [&](int64_t p) {
        const int rows = (int)min((int64_t)TT, L - p);
        if (a.bc16) {
            for (int i = tid; i < rows * (S / VB); i += NT) {
                const int t = i / (S / VB), v = (i % (S / VB)) * VB;
                ssm_cp_async<16>(rawB + t * S + v, B + at((int)(lo + p) + t, a.ldB) + v);
                ssm_cp_async<16>(rawB + (TT + t) * S + v, C + at((int)(lo + p) + t, a.ldC) + v);
            }
        } else {
            for (int i = tid; i < rows * S; i += NT) {
                const int t = i / S, v = i % S;
                rawB[i] = B[(lo + p + t) * a.ldB + v];
                rawB[TT * S + i] = C[(lo + p + t) * a.ldC + v];
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    if (L > 0) {
        stage(0, 0);
        stage_bc(0);
    }
    const f2x shift = pk2(kEx2Mean, kEx2Mean);
    const f2x later = seg == 0 ? pk2(0.0f, 0.0f) : pk2(1.0f, 1.0f);
    int buf = 0;
    for (int64_t p = 0; p < L; p += TT, buf ^= 1) {
        const int rows = (int)min((int64_t)TT, L - p);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // B and C as planes of state pairs, in fp32 (zero behind the sequence's end)
        for (int i = tid; i < 2 * TT * (S / VB); i += NT) {
            const int t = i % TT, j = i / TT;  // neighbouring threads, neighbouring tokens
            const int v = (j % (S / VB)) * VB;
            const bool isC = j >= S / VB;
            const Vec<T, VB> r = load_vec<T, VB>(rawB + ((isC ? TT : 0) + t) * S + v);
            float2* d = (isC ? sC : sB) + (v / 2) * Cf::PS + (t / K) * (K + 2) + t % K;
            if (t < rows) {
#pragma unroll
                for (int q = 0; q < VB / 2; ++q)
                    d[q * Cf::PS] = make_float2(to_f<T>(r.v[2 * q]), to_f<T>(r.v[2 * q + 1]));
            } else {
#pragma unroll
                for (int q = 0; q < VB / 2; ++q) d[q * Cf::PS] = make_float2(0.f, 0.f);
            }
        }
        if (p + TT < L) stage(p + TT, buf ^ 1);
        T* mine = raw + buf * 3 * Cf::TOK + seg * Cf::SEGROW + ch;
        f2x dl[K], u[K], y[K];  // delta and delta x in both halves
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float d = ssm_delta(a, to_f<T>(mine[Cf::TOK + k * CB]), bias), w = d * to_f<T>(mine[k * CB]);
            dl[k] = pk2(d, d);
            u[k] = pk2(w, w);
            y[k] = pk2(0.0f, 0.0f);
        }
        if (rows < TT) {  // behind the sequence's end: the state stays
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (seg * K + k >= rows) dl[k] = u[k] = pk2(0.0f, 0.0f);
        }
        __syncthreads();
        if (p + TT < L) stage_bc(p + TT);
#pragma unroll 1
        for (int np = 0; np < NP; ++np) {
            const f2x A2 = *reinterpret_cast<const f2x*>(sA + np * CB + ch);
            const f2x h0 = *reinterpret_cast<const f2x*>(sH + np * CB + ch);
            const ulonglong2* pB = reinterpret_cast<const ulonglong2*>(sB + np * Cf::PS + seg * (K + 2));
            const ulonglong2* pC = reinterpret_cast<const ulonglong2*>(sC + np * Cf::PS + seg * (K + 2));
            f2x am[K], bm[K], P, H;
#pragma unroll
            for (int k2 = 0; k2 < K / 2; ++k2) {
                const ulonglong2 b2 = pB[k2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int k = 2 * k2 + q;
                    float e0, e1;
                    up2(ffma2(dl[k], A2, shift), e0, e1);
                    am[k] = pk2(ex2(e0), ex2(e1));
                    bm[k] = fmul2(u[k], q ? b2.y : b2.x);
                    if (k == 0) {
                        P = fmul2(am[0], later);
                        H = seg == 0 ? ffma2(am[0], h0, bm[0]) : bm[0];
                    } else {
                        P = fmul2(P, am[k]);
                        H = ffma2(am[k], H, bm[k]);
                    }
                }
            }
            // inclusive scan over the segments: (P, H) o (Pp, Hp) = (P Pp, P Hp + H).  The
            // first segment's P is 0, as its H holds the carried state already; so P
            // becomes 0 in every lane that has joined it, and the lanes without an
            // earlier segment, which get their own H back, keep it.
#pragma unroll
            for (int o = 1; o < SEG; o <<= 1) {
                H = ffma2(P, __shfl_up_sync(kFullMask, H, o * CL), H);
                if (2 * o < SEG) P = fmul2(P, __shfl_up_sync(kFullMask, P, o * CL));
            }
            const f2x from = __shfl_sync(kFullMask, H, (lane - CL) & 31);  // the first segment gets the last's
            f2x h = seg == 0 ? h0 : from;
            if (seg == 0) *reinterpret_cast<f2x*>(sH + np * CB + ch) = from;
            if (a.saved != nullptr && on && (seg * K) % kSsmSave == 0 && seg * K < rows) {
                const int64_t at = a.s.first_slot(n, kSsmSave) + (p + seg * K) / kSsmSave;
                *reinterpret_cast<f2x*>(a.saved + (at * a.D + ch0) * S + 2 * np) = h;
            }
#pragma unroll
            for (int k2 = 0; k2 < K / 2; ++k2) {
                const ulonglong2 c2 = pC[k2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int k = 2 * k2 + q;
                    h = ffma2(am[k], h, bm[k]);
                    y[k] = ffma2(h, q ? c2.y : c2.x, y[k]);
                }
            }
        }
        // y in the place of x
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float y0, y1;
            up2(y[k], y0, y1);
            float o = __fmaf_rn(Dv, to_f<T>(mine[k * CB]), y0 + y1);
            if (a.z != nullptr) o *= silu(to_f<T>(mine[2 * Cf::TOK + k * CB]));
            mine[k * CB] = from_f<T>(o);
        }
        __syncthreads();
        const T* out = raw + buf * 3 * Cf::TOK;
        for (int i = tid; i < TT * (CB / V); i += NT) {
            const int t = i / (CB / V), v = (i % (CB / V)) * V;
            if (t < rows && cbase + v < cend)
                *reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.y) + at((int)(lo + p) + t, a.D) + cbase + v) =
                    load_vec<T, V>(out + (t / K) * Cf::SEGROW + (t % K) * CB + v);
        }
    }
    __syncthreads();
    for (int i = tid; i < CB * S; i += NT) {
        const int c = i / S, st = i % S;
        if (cbase + c < cend)
            a.state_out[((int64_t)n * a.D + cbase + c) * S + st] =
                reinterpret_cast<const float*>(sH)[((st / 2) * CB + c) * 2 + (st & 1)];
    }
}

// One token per sequence: bound by the state, read and written once.  A
// channel's S states lie with S / 4 lanes, one float4 each.
template <typename T, int S>
__global__ void __launch_bounds__(256) k_ssm_step(const SsmArgs a)
{
    constexpr int LN = S / 4;
    // a grid row per sequence; 256 / LN channels per block
    const int64_t n = blockIdx.y;
    const int cc = blockIdx.x * (256 / LN) + threadIdx.x / LN, q = threadIdx.x & (LN - 1);
    const bool on = cc < a.D;
    const int c = on ? cc : 0, e = a.G == 1 ? 0 : c / a.Dg;
    const int64_t i = n * a.D + c;
    const float4 h = *reinterpret_cast<const float4*>(a.state_in + i * S + 4 * q);
    const float4 A = *reinterpret_cast<const float4*>(a.A + (int64_t)c * S + 4 * q);
    const float x = to_f<T>(static_cast<const T*>(a.x)[n * a.ldx + c]);
    const float d = ssm_delta(a, to_f<T>(static_cast<const T*>(a.dt)[n * a.lddt + c]),
                              a.dt_bias != nullptr ? a.dt_bias[c] : 0.0f);
    const T* pB = static_cast<const T*>(a.B) + n * a.ldB + e * S + 4 * q;
    const T* pC = static_cast<const T*>(a.C) + n * a.ldC + e * S + 4 * q;
    float B[4], C[4];
    if (a.bc16) {
        const Vec<T, 4> vb = load_vec<T, 4>(pB), vc = load_vec<T, 4>(pC);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            B[k] = to_f<T>(vb.v[k]);
            C[k] = to_f<T>(vc.v[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            B[k] = to_f<T>(pB[k]);
            C[k] = to_f<T>(pC[k]);
        }
    }
    const float u = d * x, d2 = d * kLog2e;
    float4 o;
    o.x = __fmaf_rn(ex2(__fmaf_rn(d2, A.x, kEx2Mean)), h.x, u * B[0]);
    o.y = __fmaf_rn(ex2(__fmaf_rn(d2, A.y, kEx2Mean)), h.y, u * B[1]);
    o.z = __fmaf_rn(ex2(__fmaf_rn(d2, A.z, kEx2Mean)), h.z, u * B[2]);
    o.w = __fmaf_rn(ex2(__fmaf_rn(d2, A.w, kEx2Mean)), h.w, u * B[3]);
    float s = o.x * C[0];
    s = __fmaf_rn(o.y, C[1], s);
    s = __fmaf_rn(o.z, C[2], s);
    s = __fmaf_rn(o.w, C[3], s);
#pragma unroll
    for (int w = LN / 2; w > 0; w >>= 1) s += __shfl_xor_sync(kFullMask, s, w);
    if (!on) return;
    *reinterpret_cast<float4*>(a.state_out + i * S + 4 * q) = o;
    if (q == 0) {
        if (a.Dp != nullptr) s = __fmaf_rn(a.Dp[c], x, s);
        if (a.z != nullptr) s *= silu(to_f<T>(static_cast<const T*>(a.z)[n * a.ldz + c]));
        static_cast<T*>(a.y)[i] = from_f<T>(s);
    }
}

}  // namespace gdn

// k_qknorm.cuh -- norms of the queries' and keys' heads with the position rotation in the same
// pass, forward and backward (sm_100a).
//
//     r = (sum x^2 / n + eps)^(-1/2),  u = x r w      (n = d, or 1 for unit length)
//     the first R dimensions turn in pairs (a, b) by the angle p f_i of the token's position p:
//     a' = a cos - b sin,  b' = b cos + a sin
// and, with g = the gradient turned back and h = g w:
//     dx = r (h - x r sum(h x) r / n),  dw = sum_rows g x r
//
// One read of x (and dy), one write, q and k in one launch; with few tokens several blocks share the heads of
// each.  A row (one head of one token) lies in the registers of tpr neighbouring lanes, each with four pairs, so that a
// pair's two elements meet in one thread and turn without an exchange.  A block takes `tokens` tokens at a time and
// makes their angles once, for all heads, in shared memory: position times frequency in turns
// and in 64 bits, so that far positions keep their angle (at 10^6 tokens fp32 is off by 0.06), with the whole turns
// taken off before sincospi in fp32.
//
// Bound by the bytes, 4 (forward) and 6 (gradients) per bf16 element, and close behind by instructions: 164 warp
// instructions per two rows of 128.  16384 tokens x (16 + 16) heads of 128 bf16 with rotation take 58 us (4.6 TB/s);
// x (32 + 32) heads forward 112 and gradients 168 + 5 us (4.8 TB/s).  64 tokens x (32 + 32) take 6 us, 3001 x (7 + 3)
// heads of 90 fp32 12 us: latency.
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
    int32_t ring;       // where the ring starts in shared memory
    float* part;        // backward: [grid][2][d] sums of dw, or null
};

constexpr int kQkThreads = 256;
__host__ __device__ constexpr int qk_rows(bool bwd, int esize) { return bwd || esize == 4 ? 2 : 4; }  // rows of a thread in flight
__host__ __device__ constexpr int qk_resident(bool bwd, bool vec) { return bwd || !vec ? 2 : 3; }  // blocks per SM

// A thread's four neighbouring pairs of a row: the elements a(i) and b(i), i < 4.  INTER: (2 p, 2 p + 1), else
// (p, p + R / 2), and behind the rotated ones any two that are left.
template <bool INTER>
struct QkPairs {
    int first, n, R2;
    __device__ __forceinline__ QkPairs(const QkArgs& a, int lane) : first(lane * 4), n(a.d / 2), R2(a.rot / 2) {}
    __device__ __forceinline__ bool has(int i) const { return first + i < n; }
    __device__ __forceinline__ int a(int i) const
    {
        const int p = first + i;
        return INTER ? 2 * p : (p < R2 ? p : p + R2);
    }
    __device__ __forceinline__ int b(int i) const
    {
        const int p = first + i;
        return INTER ? 2 * p + 1 : (p < R2 ? p + R2 : p + n);
    }
};

// A thread's share of a row, as it lies in memory: two accesses of four elements (VEC: all of its pairs or none are
// there), or one element at a time.  The sums, and with them the bits, are the same.
template <typename T, bool VEC, bool INTER>
struct QkRow {
    Vec<T, 4> lo, hi;
    __device__ __forceinline__ void load(const T* row, const QkPairs<INTER>& q, int ea, int eb)
    {
        if constexpr (VEC) {
            lo = load_vec<T, 4>(row + ea);
            hi = load_vec<T, 4>(row + eb);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                T& x = INTER ? (i < 2 ? lo.v[2 * i] : hi.v[2 * i - 4]) : lo.v[i];
                T& y = INTER ? (i < 2 ? lo.v[2 * i + 1] : hi.v[2 * i - 3]) : hi.v[i];
                x = q.has(i) ? row[q.a(i)] : from_f<T>(0.0f);
                y = q.has(i) ? row[q.b(i)] : from_f<T>(0.0f);
            }
        }
    }
    // (a0, a1), (a2, a3) and (b0, b1), (b2, b3), widened
    __device__ __forceinline__ void get(f2x (&va)[2], f2x (&vb)[2]) const
    {
        if constexpr (INTER) {
            va[0] = pk2(to_f<T>(lo.v[0]), to_f<T>(lo.v[2])), va[1] = pk2(to_f<T>(hi.v[0]), to_f<T>(hi.v[2]));
            vb[0] = pk2(to_f<T>(lo.v[1]), to_f<T>(lo.v[3])), vb[1] = pk2(to_f<T>(hi.v[1]), to_f<T>(hi.v[3]));
        } else {
            va[0] = pbits<T, 4>(lo, 0), va[1] = pbits<T, 4>(lo, 1);
            vb[0] = pbits<T, 4>(hi, 0), vb[1] = pbits<T, 4>(hi, 1);
        }
    }
    __device__ static __forceinline__ void store(T* row, const QkPairs<INTER>& q, int ea, int eb, const f2x (&va)[2], const f2x (&vb)[2])
    {
        float x[4], y[4];
        up2(va[0], x[0], x[1]), up2(va[1], x[2], x[3]);
        up2(vb[0], y[0], y[1]), up2(vb[1], y[2], y[3]);
        if constexpr (VEC) {
            if constexpr (INTER) {
                const float l[4] = {x[0], y[0], x[1], y[1]}, h[4] = {x[2], y[2], x[3], y[3]};
                store_vec<T, 4>(row + ea, l);
                store_vec<T, 4>(row + eb, h);
            } else {
                store_vec<T, 4>(row + ea, x);
                store_vec<T, 4>(row + eb, y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q.has(i)) {
                    row[q.a(i)] = from_f<T>(x[i]);
                    row[q.b(i)] = from_f<T>(y[i]);
                }
        }
    }
};

// Four consecutive floats as two pairs; the address is 16-byte aligned.
__device__ __forceinline__ void qk_four(const float* p, f2x (&v)[2])
{
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = pk2(f.x, f.y), v[1] = pk2(f.z, f.w);
}

// A thread's own pieces of the rows that it will work on next, in a ring in shared memory that cp.async fills, as
// NormRing: the next rows are under way through the sums of these, without registers or barriers.
constexpr int kQkAhead = 2;  // turns ahead
template <typename T, typename G, int U, bool BWD>
struct QkRing {
    static constexpr int PX = 4 * (int)sizeof(T), PG = 4 * (int)sizeof(G);     // bytes of a piece of x, and of its gradient
    static constexpr int ROW = 2 * (PX + (BWD ? PG : 0)) * kQkThreads;
    static constexpr size_t BYTES = (size_t)kQkAhead * U * ROW;
    unsigned char* base;
    template <int TENSOR>
    __device__ __forceinline__ unsigned char* at(int turn, int u, int piece) const
    {
        constexpr int P = TENSOR ? PG : PX;
        // (one product for a thread's place where the pieces are alike: the gradients' registers are all taken)
        if constexpr (PX == PG) return base + ((((turn * U + u) * (BWD ? 2 : 1) + TENSOR) * 2 + piece) * kQkThreads + threadIdx.x) * P;
        return base + (turn * U + u) * ROW + (TENSOR * 2 * PX + piece * P) * kQkThreads + threadIdx.x * P;
    }
    template <int TENSOR>
    __device__ __forceinline__ void copy(int turn, int u, int piece, const void* src) const
    {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((unsigned)__cvta_generic_to_shared(at<TENSOR>(turn, u, piece))),
                     "l"(src), "n"(TENSOR ? PG : PX) : "memory");
    }
    template <int TENSOR, typename R>
    __device__ __forceinline__ void get(int turn, int u, R& row) const
    {
        row.lo = *reinterpret_cast<const decltype(row.lo)*>(at<TENSOR>(turn, u, 0));
        row.hi = *reinterpret_cast<const decltype(row.hi)*>(at<TENSOR>(turn, u, 1));
    }
};

// BWD: the gradients, from those of the outputs in type G: the recurrence's own gradients are fp32, whatever its inputs, and a pass
// of their own to bf16 would cost more than their bytes here (16384 tokens x (32 + 32) heads of 128: 197 us, with the casts 293).
// Registers: 128 for the gradients, which bf16 rows on their alignment just fit; fp32 rows or fp32 gradients spill 4 to 24 bytes per
// thread and rows off their alignment 160 to 284 (16384 x (16 + 16) heads of 128: 207 us in place of about 90).
template <typename T, typename G, bool VEC, bool INTER, bool BWD>
__global__ void __launch_bounds__(kQkThreads, qk_resident(BWD, VEC)) k_qk_norm(const QkArgs a)
{
    constexpr int U = qk_rows(BWD, sizeof(T));
    using Row = QkRow<T, VEC, INTER>;
    using Grad = QkRow<G, VEC, INTER>;
    extern __shared__ __align__(16) unsigned char qk_smem[];
    let_next_start();
    after_previous();
    // cosines [tokens][span] and sines, 1 and 0 behind the rotated pairs; span: the pairs of all lanes
    float* cs = reinterpret_cast<float*>(qk_smem);
    const int tpr = a.tpr, lane = threadIdx.x & (tpr - 1), slot = threadIdx.x / tpr, slots = kQkThreads / tpr;
    const int R2 = a.rot / 2, span = tpr * 4, half = a.tokens * span;
    const QkPairs<INTER> pairs(a, lane);
    float* ws = cs + (R2 > 0 ? 2 * half : 0);  // weights [2][2][span]: those of the a's, then of the b's
    const bool mine = pairs.has(0);
    // VEC: where the two accesses start; lanes without a pair read the row's first elements, which count for nothing
    const int ea = !mine ? 0 : INTER ? 2 * pairs.first : pairs.a(0), eb = !mine ? 0 : INTER ? 2 * pairs.first + 4 : pairs.b(0);
    for (int i = threadIdx.x; i < 2 * span; i += kQkThreads) {
        const int kind = i / span, p = i - kind * span;
        const QkPairs<INTER> q(a, p / 4);
        const bool in = a.w[kind] != nullptr && q.has(p % 4);
        ws[(2 * kind) * span + p] = in ? load_w(a.w[kind], a.w_bf16, q.a(p % 4)) : 1.0f;
        ws[(2 * kind + 1) * span + p] = in ? load_w(a.w[kind], a.w_bf16, q.b(p % 4)) : 1.0f;
    }
    __syncthreads();
    const bool weighted = a.w[0] != nullptr || a.w[1] != nullptr;
    // this thread's columns of dw: of the kind that is worked on, and of the other one
    f2x da[2], db[2], oa[2], ob[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) da[i] = db[i] = oa[i] = ob[i] = pk2(0.0f, 0.0f);

    const int64_t tiles = (a.T + a.tokens - 1) / a.tokens;
    // this block's share of a tile's rows, in whole rounds of the slots
    auto share = [&](int all, int& begin, int& end) {
        const int n = (int)(((int64_t)all + slots * gridDim.y - 1) / (slots * gridDim.y)) * slots;
        begin = min(all, n * (int)blockIdx.y);
        end = min(all, begin + n);
    };
    // Where the thread's next rows to fetch lie: from one to the next, `slots` rows on, dt tokens and dh heads, or one token
    // more and H heads less.
    struct {
        int64_t tile, stepx, wrapx, stepg, wrapg;
        const T* px;
        const G* pg;
        int kind, r, end, h, H, dh;
    } next{};
    auto aim = [&] {  // at the first row of next.kind in next.tile
        const int64_t t0 = next.tile * a.tokens;
        const bool k = next.kind;  // (no indexed arguments: they would be copied to local memory)
        const int H = k ? a.H[1] : a.H[0], dt = slots / H;
        int begin;
        share((int)min((int64_t)a.tokens, a.T - t0) * H, begin, next.end);
        const int64_t ldx = k ? a.ldx[1] : a.ldx[0], ldg = BWD ? (k ? a.lddy[1] : a.lddy[0]) : 0;
        const int tok = (begin + slot) / H;
        next.H = H;
        next.dh = slots - dt * H;
        next.h = begin + slot - tok * H;
        next.r = begin;
        next.px = static_cast<const T*>(k ? a.x[1] : a.x[0]) + (t0 + tok) * ldx + next.h * a.d;
        next.stepx = dt * ldx + next.dh * a.d, next.wrapx = ldx - (int64_t)H * a.d;
        if constexpr (BWD) {
            next.pg = static_cast<const G*>(k ? a.dy[1] : a.dy[0]) + (t0 + tok) * ldg + next.h * a.d;
            next.stepg = dt * ldg + next.dh * a.d, next.wrapg = ldg - (int64_t)H * a.d;
        }
    };
    auto advance = [&] {
        next.px += next.stepx;
        if constexpr (BWD) next.pg += next.stepg;
        if (next.dh != 0) {
            next.h += next.dh;
            if (next.h >= next.H) {
                next.h -= next.H;
                next.px += next.wrapx;
                if constexpr (BWD) next.pg += next.wrapg;
            }
        }
    };
    auto skip = [&] {  // over what has no rows (left)
        while (next.tile < tiles && next.r >= next.end) {
            if (next.kind) next.tile += gridDim.x;
            next.kind ^= 1;
            if (next.tile < tiles) aim();
        }
    };
    const QkRing<T, G, U, BWD> ring{qk_smem + a.ring};
    int turn = 0;  // of the ring
    auto fetch = [&](int turn) {
        if (next.tile < tiles) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (next.r + u * slots + slot < next.end) {
                    ring.template copy<0>(turn, u, 0, next.px + ea);
                    ring.template copy<0>(turn, u, 1, next.px + eb);
                    if constexpr (BWD) {
                        ring.template copy<1>(turn, u, 0, next.pg + ea);
                        ring.template copy<1>(turn, u, 1, next.pg + eb);
                    }
                }
                advance();
            }
            next.r += U * slots;
            skip();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    next.tile = blockIdx.x;
    next.kind = 0;
    if (next.tile < tiles) {
        aim();
        skip();
    }
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kQkAhead; ++i) fetch(i);
    }
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t t0 = tile * a.tokens;
        const int nt = (int)min((int64_t)a.tokens, a.T - t0);
        if (R2 > 0) {
            __syncthreads();  // the last tile's angles have been read
            for (int i = threadIdx.x; i < nt * span; i += kQkThreads) {
                const int t = i / span, p = i - t * span;
                float s = 0.0f, c = 1.0f;
                if (p < R2) {
                    const double turns = (double)a.pos[t0 + t] * ((double)a.freq[p] * 0.15915494309189533577);
                    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
                }
                cs[i] = c;
                cs[half + i] = s;
            }
            __syncthreads();
        }
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            f2x wa[2], wb[2];
            qk_four(ws + 2 * kind * span + pairs.first, wa);
            qk_four(ws + (2 * kind + 1) * span + pairs.first, wb);
            const int H = kind ? a.H[1] : a.H[0], dt = slots / H, dh = slots - dt * H;
            int begin, rows;
            share(nt * H, begin, rows);
            const int tok0 = (begin + slot) / H;
            int h = begin + slot - tok0 * H, at = tok0 * span + pairs.first;  // the head and the angles of this thread's next row
            T* po = static_cast<T*>(kind ? a.out[1] : a.out[0]) + (t0 * H + begin + slot) * (int64_t)a.d;
            const int64_t stepo = (int64_t)slots * a.d;
            auto some = [&](auto all, int r0) {  // U rows of every thread; WHOLE: all of them are there
                constexpr bool WHOLE = decltype(all)::value;
                Row x[U];
                [[maybe_unused]] Grad g[BWD ? U : 1];
                int ang[U];
                bool on[U];
                if constexpr (VEC) asm volatile("cp.async.wait_group %0;" ::"n"(kQkAhead - 1) : "memory");
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    on[u] = WHOLE || r0 + u * slots + slot < rows;
                    ang[u] = at;
                    if constexpr (!VEC) {
                        if (on[u]) {
                            x[u].load(next.px, pairs, ea, eb);
                            if constexpr (BWD) g[u].load(next.pg, pairs, ea, eb);
                        }
                        advance();
                    }
                    at += dt * span;
                    if (dh != 0) {
                        h += dh;
                        if (h >= H) h -= H, at += span;
                    }
                }
                if constexpr (!VEC) {
                    next.r += U * slots;
                    skip();
                }
                float ss[U];
                [[maybe_unused]] float sg[BWD ? U : 1];
                [[maybe_unused]] f2x ga[BWD ? U : 1][2], gb[BWD ? U : 1][2];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    ss[u] = 0.0f;
                    if constexpr (BWD) sg[u] = 0.0f;
                    if (on[u]) {
                        f2x va[2], vb[2];
                        if constexpr (VEC) ring.template get<0>(turn, u, x[u]);
                        x[u].get(va, vb);
                        ss[u] = psum(pfma(va[0], va[0], pfma(va[1], va[1], pfma(vb[0], vb[0], pmul(vb[1], vb[1])))));
                        if constexpr (BWD) {
                            if constexpr (VEC) ring.template get<1>(turn, u, g[u]);
                            g[u].get(ga[u], gb[u]);
                            if (R2 > 0) {  // turned back
                                f2x c[2], s[2];
                                qk_four(cs + ang[u], c);
                                qk_four(cs + half + ang[u], s);
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const f2x p = ga[u][i], q = gb[u][i];
                                    ga[u][i] = pfma(p, c[i], pmul(q, s[i]));
                                    gb[u][i] = pfma(pmul(p, pk2(-1.0f, -1.0f)), s[i], pmul(q, c[i]));
                                }
                            }
                            f2x acc = pmul(pmul(ga[u][0], wa[0]), va[0]);
                            acc = pfma(pmul(ga[u][1], wa[1]), va[1], acc);
                            acc = pfma(pmul(gb[u][0], wb[0]), vb[0], acc);
                            sg[u] = psum(pfma(pmul(gb[u][1], wb[1]), vb[1], acc));
                            if (!mine) sg[u] = 0.0f;
                        }
                        if (!mine) ss[u] = 0.0f;
                    }
                }
                auto fold = [&](int o) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        ss[u] += __shfl_xor_sync(kFullMask, ss[u], o);
                        if constexpr (BWD) sg[u] += __shfl_xor_sync(kFullMask, sg[u], o);
                    }
                };
                if (tpr > 16) fold(16);
                if (tpr > 8) fold(8);
                if (tpr > 4) fold(4);
                if (tpr > 2) fold(2);
                if (tpr > 1) fold(1);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (on[u]) {
                        const float rr = inv_sqrt(__fmaf_rn(ss[u], a.inv_n, a.eps));
                        const f2x r2 = pk2(rr, rr);
                        f2x va[2], vb[2];
                        if constexpr (VEC) {
                            asm volatile("" ::: "memory");  // read again: it need not wait in registers
                            ring.template get<0>(turn, u, x[u]);
                        } else {
                            keep_packed(x[u].lo);
                            keep_packed(x[u].hi);
                        }
                        x[u].get(va, vb);
                        if constexpr (BWD) {
                            // as in layer norm, no power of r is formed: x r is again about 1
                            const float c = -(sg[u] * rr * a.inv_n);
                            const f2x c2 = pk2(c, c);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const f2x na = pmul(va[i], r2), nb = pmul(vb[i], r2);
                                da[i] = pfma(ga[u][i], na, da[i]);
                                db[i] = pfma(gb[u][i], nb, db[i]);
                                va[i] = pmul(r2, pfma(na, c2, pmul(ga[u][i], wa[i])));
                                vb[i] = pmul(r2, pfma(nb, c2, pmul(gb[u][i], wb[i])));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                va[i] = pmul(va[i], r2);
                                vb[i] = pmul(vb[i], r2);
                                if (weighted) {
                                    va[i] = pmul(va[i], wa[i]);
                                    vb[i] = pmul(vb[i], wb[i]);
                                }
                            }
                            if (R2 > 0) {
                                f2x c[2], s[2];
                                qk_four(cs + ang[u], c);
                                qk_four(cs + half + ang[u], s);
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const f2x p = va[i], q = vb[i];
                                    va[i] = pfma(pmul(q, pk2(-1.0f, -1.0f)), s[i], pmul(p, c[i]));
                                    vb[i] = pfma(p, s[i], pmul(q, c[i]));
                                }
                            }
                        }
                        if (mine) Row::store(po + u * stepo, pairs, ea, eb, va, vb);
                    }
                }
                po += U * stepo;
                if constexpr (VEC) {
                    fetch(turn);  // behind the last use of what lies there
                    turn = turn + 1 == kQkAhead ? 0 : turn + 1;
                }
            };
            // the same turns for every thread: the sums are shuffles
            int r0 = begin;
            for (; r0 + slots * U <= rows; r0 += slots * U) some(std::true_type{}, r0);
            if (r0 < rows) some(std::false_type{}, r0);
            if constexpr (BWD) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f2x t = da[i];
                    da[i] = oa[i], oa[i] = t;
                    t = db[i];
                    db[i] = ob[i], ob[i] = t;
                }
            }
        }
    }
    if constexpr (BWD) {
        if (a.part == nullptr) return;
        // dw: the rows of a warp by shuffles, then the warps in order
        float* red = cs;  // [8][d]
        float* part = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.d;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            float x[4], y[4];
            up2(kind ? oa[0] : da[0], x[0], x[1]), up2(kind ? oa[1] : da[1], x[2], x[3]);
            up2(kind ? ob[0] : db[0], y[0], y[1]), up2(kind ? ob[1] : db[1], y[2], y[3]);
            for (int o = 16; o >= tpr; o >>= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] += __shfl_xor_sync(kFullMask, x[i], o);
                    y[i] += __shfl_xor_sync(kFullMask, y[i], o);
                }
            __syncthreads();
            if ((threadIdx.x & 31) < tpr) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (pairs.has(i)) {
                        red[(threadIdx.x >> 5) * a.d + pairs.a(i)] = x[i];
                        red[(threadIdx.x >> 5) * a.d + pairs.b(i)] = y[i];
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

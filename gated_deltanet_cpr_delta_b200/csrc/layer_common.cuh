// layer_common.cuh -- device helpers shared by the layer operators around the
// recurrence (k_conv.cuh, k_norm.cuh, k_ssm.cuh, k_ssm_bwd.cuh).
//
// Unlike the CPR path these operators have no bitwise contract between their
// entry points.  Their sums are fp32 in a fixed order, without atomics, so
// repeated calls give the same bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "schedule.cuh"

namespace gdn {

// Element types: float, or bf16 widened exactly on load and rounded to
// nearest-even once, on store.
template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements as one memory access (V * sizeof(T) in {2, 4, 8, 16}).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p)
{
    return *reinterpret_cast<const Vec<T, V>*>(p);
}

// Two bf16 rounded at once.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* x)
{
    Vec<T, V> r;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t* u = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) u[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = from_f<T>(x[i]);
    }
    *reinterpret_cast<Vec<T, V>*>(p) = r;
}

// Pairs of fp32 values in one packed register (f2x), or single ones where a
// thread has no neighbour (V = 1): the same code for both.
template <int V>
struct Lanes {
    using type = f2x;
    static constexpr int N = V / 2;
};
template <>
struct Lanes<1> {
    using type = float;
    static constexpr int N = 1;
};
__device__ __forceinline__ f2x fadd2(f2x a, f2x b)
{
    f2x d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2x padd(f2x a, f2x b) { return fadd2(a, b); }
__device__ __forceinline__ float padd(float a, float b) { return a + b; }
__device__ __forceinline__ f2x pmul(f2x a, f2x b) { return fmul2(a, b); }
__device__ __forceinline__ float pmul(float a, float b) { return a * b; }
__device__ __forceinline__ f2x pfma(f2x a, f2x b, f2x c) { return ffma2(a, b, c); }
__device__ __forceinline__ float pfma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ float psum(f2x a)
{
    float x, y;
    up2(a, x, y);
    return x + y;
}
__device__ __forceinline__ float psum(float a) { return a; }
template <int V>
__device__ __forceinline__ typename Lanes<V>::type pset(float x)
{
    if constexpr (V == 1) return x;
    else return pk2(x, x);
}
// element or pair i of V elements of type T, widened
template <typename T, int V>
__device__ __forceinline__ typename Lanes<V>::type pget(const Vec<T, V>& r, int i)
{
    if constexpr (V == 1) {
        return to_f<T>(r.v[0]);
    } else {
        return pk2(to_f<T>(r.v[2 * i]), to_f<T>(r.v[2 * i + 1]));
    }
}
// The same by a shift and a mask of the packed word.  Layer norm, which holds rows packed
// and widens them where they are used, is a fifth faster with it (59 against 75 us), the
// convolution, which widens what has just arrived, a fifth slower (96 against 77 us).
template <typename T, int V>
__device__ __forceinline__ typename Lanes<V>::type pbits(const Vec<T, V>& r, int i)
{
    if constexpr (V > 1 && sizeof(T) == 2) {
        const uint32_t u = reinterpret_cast<const uint32_t*>(&r)[i];
        return pk2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
        return pget<T, V>(r, i);
    }
}
template <typename T, int V>
__device__ __forceinline__ void pstore(T* p, const typename Lanes<V>::type* x)
{
    float o[V];
    if constexpr (V == 1) o[0] = x[0];
    else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) up2(x[i], o[2 * i], o[2 * i + 1]);
    }
    store_vec<T, V>(p, o);
}

// V floats of shared memory, 16 bytes at a time where V allows
template <int V>
__device__ __forceinline__ void put_row(float* p, const float (&x)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = x[i];
    }
}
template <int V>
__device__ __forceinline__ void get_row(const float* p, float (&x)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p[i];
    }
}

// Weights and biases may be fp32 or bf16 whatever the tokens are.
__device__ __forceinline__ float load_w(const void* w, int bf16, int64_t i)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

// n consecutive weights from element i on, in accesses as wide as n elements and the address allow
template <int N>
__device__ __forceinline__ void load_ws(const void* w, int bf16, int64_t i, float (&x)[N])
{
    auto run = [&](auto* p) {
        using WT = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
        constexpr int B = N * sizeof(WT);  // bytes
        constexpr int A = B % 16 == 0 ? 16 : B % 8 == 0 ? 8 : B % 4 == 0 ? 4 : (int)sizeof(WT), E = A / (int)sizeof(WT);
        if ((reinterpret_cast<uintptr_t>(p) & (A - 1)) == 0) {
#pragma unroll
            for (int j = 0; j < N / E; ++j) {
                const Vec<WT, E> v = load_vec<WT, E>(p + j * E);
#pragma unroll
                for (int k = 0; k < E; ++k) x[j * E + k] = to_f<WT>(v.v[k]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = to_f<WT>(p[j]);
        }
    };
    if (bf16) run(static_cast<const __nv_bfloat16*>(w) + i);
    else run(static_cast<const float*>(w) + i);
}

// The packed batch: sequence n holds rows [lo(n), hi(n)).  Offsets come from
// device memory and are clamped to [0, T], so that no value of them makes an
// access leave the tensors.  cu == nullptr: one sequence of T rows.
struct Seqs {
    const int32_t* cu;
    int32_t N;
    int64_t T;
    __device__ __forceinline__ int64_t at(int n) const
    {
        if (cu == nullptr) return n == 0 ? 0 : T;
        const int64_t c = cu[n];
        return c < 0 ? 0 : (c > T ? T : c);
    }
    __device__ __forceinline__ int64_t lo(int n) const { return at(n); }
    __device__ __forceinline__ int64_t hi(int n) const
    {
        const int64_t a = at(n), b = at(n + 1);
        return b < a ? a : b;
    }
    // The last sequence that starts at or before row t; -1 if none does.
    __device__ __forceinline__ int find(int64_t t) const
    {
        int a = -1, b = N;  // lo(a) <= t < lo(b)
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (at(m) <= t) a = m;
            else b = m;
        }
        return a;
    }
    // Chunks of `len` tokens per sequence, numbered without a table: chunk c of
    // sequence n is slot lo(n) / len + n + c.  Slots are distinct, because
    // floor((a + L) / len) - floor(a / len) + 1 >= ceil(L / len), and lie below
    // T / len + N.
    __device__ __forceinline__ int64_t first_slot(int n, int64_t len) const { return lo(n) / len + n; }
    __device__ __forceinline__ int find_slot(int64_t slot, int64_t len) const
    {
        int a = 0, b = N;
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (first_slot(m, len) <= slot) a = m;
            else b = m;
        }
        return a;
    }
};

// One block of a kernel checks the device offsets (0 <= cu[0], non-decreasing,
// cu[N] <= T) and records the first error it sees.
__device__ __forceinline__ void check_seqs(const Seqs& s, int32_t* status)
{
    if (status == nullptr || s.cu == nullptr) return;
    for (int n = threadIdx.x; n <= s.N; n += blockDim.x) {
        const int64_t c = s.cu[n];
        const bool bad = c < 0 || c > s.T || (n > 0 && c < s.cu[n - 1]);
        if (bad) atomicCAS(status, GDN_OK, GDN_ERR_DEVICE_INPUT);
    }
}

// 2^x in one instruction.  Measured against the exact value over [-10, -1e-5]:
// relative error at most 1.5e-7, 3e-8 to 6e-8 rms, and too small by 6e-9 (near 0), 1.2e-8
// to 2.6e-8 (from -0.001 to -1) and 5e-8 (below) in the mean.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// A state that decays slowly multiplies thousands of such factors close to 1, whose mean
// error then adds up.  The decays take 2^(x + kEx2Mean), which costs nothing as the
// exponent is a product already: it raises a factor by 1.6e-8, so that the mean error is at most
// 1e-8 where it matters; x = 0 still gives exactly 1.
constexpr float kEx2Mean = 2.3e-8f;

// 1 / x in one instruction, off by at most one unit; 0 for x above 2^126
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + ex2(-kLog2e * v)); }

// v * sigmoid(v) and its derivative
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ float silu_grad(float v)
{
    const float s = sigmoid(v);
    return s * __fmaf_rn(v, 1.0f - s, 1.0f);
}

// The smaller of two values; not a number if one of them is not
__device__ __forceinline__ float min_nan(float a, float b)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1], with log1p(e) = e P(e).  P is a polynomial
// of degree 9 by the exchange algorithm; as rounded to fp32 it is off by at most 3.3e-8 on [0, 1].
// Nine multiply-adds in place of the library's log1pf, which took a quarter of the scan's instructions.
// e = 2^t e^r, where t = -|v| log2 e is rounded and r = -|v| - t ln 2, exact but for ln 2's own rounding, is
// what that left: without it e^-|v|, and with it the value, is off by |v| / 2 units more.  Off by
// at most 9 units of 2^-24 of its value for v above -20 (measured on 262144 values of [-20, 5]: 3.9);
// below 2^-126 it is 0.
__device__ __forceinline__ float softplus(float v)
{
    const float w = min_nan(fabsf(v), 128.0f);  // e is 0 there: r stays finite where v is not
    const float t = -kLog2e * w;
    float e = ex2(t);
    e = __fmaf_rn(e, __fmaf_rn(t, -0.6931471805599453f, -w), e);
    float p = -0.0032440251670777798f;
    p = __fmaf_rn(p, e, 0.01985146291553974f);
    p = __fmaf_rn(p, e, -0.05695953592658043f);
    p = __fmaf_rn(p, e, 0.10603655129671097f);
    p = __fmaf_rn(p, e, -0.15305592119693756f);
    p = __fmaf_rn(p, e, 0.1967593878507614f);
    p = __fmaf_rn(p, e, -0.24954134225845337f);
    p = __fmaf_rn(p, e, 0.3332996368408203f);
    p = __fmaf_rn(p, e, -0.4999990165233612f);
    p = __fmaf_rn(p, e, 1.0f);
    return __fmaf_rn(p, e, fmaxf(v, 0.0f));
}

// Column sums out[map(m)] = sum_r in[r][m], r < R, m < M, in a fixed order: 8
// row slices per block, each summed in ascending rows, then joined in order.
// OutMap: m -> pointer to write (may be nullptr: not wanted).
template <typename OutMap>
__global__ void __launch_bounds__(256) k_colsum(const float* __restrict__ in, int64_t R, int64_t M, OutMap out)
{
    __shared__ float part[8][32];
    const int64_t m = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (m < M) {
#pragma unroll 8
        for (int64_t r = threadIdx.y; r < R; r += 8) s += in[r * M + m];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && m < M) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
        out(m, s);
    }
}

}  // namespace gdn

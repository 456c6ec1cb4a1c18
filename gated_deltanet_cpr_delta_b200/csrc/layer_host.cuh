// layer_host.cuh -- what the host sides of the layer operators share (layer_ops.cu, block_ops.cu,
// glu_ops.cu): checks of addresses, strides and overlaps, and of launches.
#pragma once

#include "gdn_cpr.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

namespace {

constexpr size_t kAlign = 256;
// The kernels count rows, the columns of the norm and the channels of the scan, and a block's worth beyond
// the end, in 32 bits.
constexpr int64_t kMaxRows = INT32_MAX - 4096;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(gdn_dtype_t t) { return t == GDN_F32 || t == GDN_BF16; }
size_t esize(gdn_dtype_t t) { return t == GDN_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool launched() { return cudaGetLastError() == cudaSuccess; }

// Shared memory beyond the 48 KB that every launch may have.  The limit is the kernel's, not the launch's: another thread's call of
// the same kernel may set it between this call's setting and its launch, so every call of a kernel sets the same value: all that the
// device gives, but for 1 KB of static shared memory, which no kernel here that varies its size passes.
constexpr int kMostSmem = 226 * 1024;
template <typename K>
bool raise_smem(K* kernel, size_t bytes)
{
    return bytes <= 48 * 1024 || (bytes <= kMostSmem &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) == cudaSuccess);
}
// For a kernel that takes the same number of bytes in every launch (and may hold more static shared memory).
template <size_t BYTES, typename K>
bool raise_smem(K* kernel)
{
    return BYTES <= 48 * 1024 ||
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BYTES) == cudaSuccess;
}

// Launches a kernel that calls after_previous(): its blocks may start, and get ready, while the kernel before it still runs
// (the gated block's step of 8 x 512 x 1024 takes 31 us in place of 39, of 500 x 701 x 1501 69 and 79).
// cluster: blocks of a cluster, 0 where the kernel states it.
template <typename... P, typename... A>
bool launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st, A&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...) == cudaSuccess && launched();
}

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return 0;
    return sms;
}

// The bytes of a [rows, width] tensor whose rows are `stride` elements apart.
struct Span {
    uintptr_t lo = 0, hi = 0;      // from the first row's start to the last row's end; empty: lo == hi
    size_t step = 0, width = 0;    // bytes between rows, and of a row
    Span(const void* p, int64_t rows, int64_t stride, int64_t row, size_t esz)
    {
        if (p == nullptr || rows <= 0 || row <= 0) return;
        lo = reinterpret_cast<uintptr_t>(p);
        step = (size_t)stride * esz;
        width = (size_t)row * esz;
        hi = lo + (size_t)(rows - 1) * step + width;
    }
    Span(const void* p, int64_t n, size_t esz) : Span(p, 1, n, n, esz) {}
    // Whether a dense tensor o shares bytes with it: its rows, not the room between them.
    bool hits(const Span& o) const
    {
        if (lo == hi || o.lo == o.hi || lo >= o.hi || o.lo >= hi) return false;
        // the first row that ends behind o's start
        const size_t k = o.lo < lo + width ? 0 : (o.lo - lo - width) / step + 1;
        return lo + k * step < o.hi;
    }
};

// Whether an output (all dense) shares bytes with an input or with another output.
bool overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (i.hits(*o)) return true;
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (o->hits(*q)) return true;
    }
    return false;
}

// 16-byte accesses: the row's address, stride and width are multiples of 16 bytes.
bool wide(const void* p, int64_t stride, int64_t width, gdn_dtype_t t)
{
    const int64_t v = 16 / (int64_t)esize(t);
    return p == nullptr || (aligned(p, 16) && stride % v == 0 && width % v == 0);
}

// Whether every row starts at, and consists of, whole groups of v elements.
bool groups(const void* p, int64_t stride, int64_t width, gdn_dtype_t t, int64_t v)
{
    return aligned(p, v * esize(t)) && stride % v == 0 && width % v == 0;
}

bool rows_ok(const void* p, int64_t stride, int64_t width, gdn_dtype_t t)
{
    return p != nullptr && stride >= width && stride <= INT32_MAX && aligned(p, esize(t));
}

}  // namespace

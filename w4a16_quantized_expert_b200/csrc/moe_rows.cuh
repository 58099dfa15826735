// moe_rows.cuh -- rows of 16- and 32-bit elements: vector loads, conversions to and from
// fp32, shared by the token-sorting and adapter kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "moe_device.cuh"

namespace moe {

// 8 consecutive elements of a row as they sit in memory (16 bytes of 16-bit, 32 of fp32)
template <typename T>
struct Vec8 {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T *p)
{
    Vec8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const Vec8<T> &r)
{
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = r.v[i];
}

__device__ __forceinline__ void to_f32(const Vec8<__half> &r, float (&f)[8])
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

__device__ __forceinline__ void to_f32(const Vec8<__nv_bfloat16> &r, float (&f)[8])
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // a bf16 is the high half of its fp32
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void to_f32(const Vec8<float> &r, float (&f)[8])
{
    const float *p = reinterpret_cast<const float *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = p[i];
}

// fp32 -> the row's type, rounded to nearest even
template <typename T>
__device__ __forceinline__ T from_f32(float f);
template <>
__device__ __forceinline__ __half from_f32<__half>(float f) { return __float2half_rn(f); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float f) { return __float2bfloat16_rn(f); }
template <>
__device__ __forceinline__ float from_f32<float>(float f) { return f; }

__device__ __forceinline__ float f32_of(__half v) { return __half2float(v); }
__device__ __forceinline__ float f32_of(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float f32_of(float v) { return v; }

template <typename T>
__device__ __forceinline__ Vec8<T> pack8(const float (&f)[8])
{
    Vec8<T> r;
    T *p = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(f[i]);
    return r;
}

// launches with the programmatic-serialisation attribute: the kernel may start while its
// predecessor on the stream drains, and waits for it (pdl_wait) before touching memory
struct ChainLaunch {
    dim3 grid;
    int threads;
    size_t smem;
    int cluster;   // CTAs (x) of a cluster
    cudaStream_t stream;
};

template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kernel)(KArgs...), const ChainLaunch &l, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = l.grid;
    cfg.blockDim = dim3(l.threads);
    cfg.dynamicSmemBytes = l.smem;
    cfg.stream = l.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = l.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = l.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// lets a kernel take all the dynamic shared memory that the device's opt-in limit leaves
// beside its static shared memory (once per device, when a handle is created)
template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...))
{
    cudaFuncAttributes a;
    int dev = 0, limit = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&limit, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, limit - (int)a.sharedSizeBytes);
}

// A stable sort of n small keys (moe_sort.cu): positions of the keys' entries when the
// entries are grouped by key, every group starting at a multiple of `align`.
struct SortParams {
    const int32_t *key;   // [n] in [0, E); other values go to none_bin, or nowhere
    int n, E, align;
    int none_bin;         // bin of the entries with key -1, or -1: they get position -1
    int32_t *counts;      // optional [E]
    int32_t *seg;         // [E + 1] first position of each group
    int32_t *row_of;      // optional [n] position of each entry
    int32_t *entry_of;    // optional: entry at each position, -1 in the padding of a group
    int32_t *tile_bin;    // optional [max_tiles]: bin of each `align` positions, -1 behind the last
    int max_tiles;
    int32_t *order;       // optional [E - 1]: the bins but the last, largest first (E <= 129)
    unsigned *zero;       // optional: n_zero words to clear
    int n_zero;
    int32_t *hist;        // scratch [ceil(n / kSortChunk)][E] (unused when n <= kSortChunk)
    int *status;
};

constexpr int kSortChunk = 2048;   // entries per CTA of the sort
cudaError_t launch_sort(const SortParams &p, cudaStream_t s);

}  // namespace moe

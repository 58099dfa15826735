// moe_adapters.cu -- low-rank adapters of many requests beside a shared projection, and
// their gradients: kernels and entry points.
#include "moe_internal.h"
#include "moe_rows.cuh"

#include <algorithm>
#include <new>

// the opaque handle
struct moe_adapters {
    moe_adapters_desc desc;
    moe_adapters_weights w;
    int *d_status;
    int device;
    int num_sms;
};

namespace moe {
namespace {

constexpr int kAdThreads = 128;

struct AdParams {
    const void *x, *dy;          // [T][K], [T][N] of the pool's type
    const void *a, *b;
    const float *scaling;
    const int32_t *rank, *adapter_of;
    const void *y_in;
    void *y;
    const float *zr;             // z read
    float *z;                    // z or dz written
    float *out;                  // da or db
    long long ldx, lddy, ldy_in, ldy;
    int T, K, N, R, n, accumulate;
    int *status;
};

__device__ __forceinline__ int adapter_at(const AdParams &p, int t)
{
    const int a = p.adapter_of[t];
    if (a >= 0 && a < p.n) return a;
    if (a != -1) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
    return -1;
}

__device__ __forceinline__ int rank_of(const AdParams &p, int a)
{
    if (!p.rank) return p.R;
    const int r = p.rank[a];
    if (r >= 0 && r <= p.R) return r;
    record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
    return 0;
}

// z[t][j] = sum_k x[t][k] A[j][k] (kGrad: dz[t][j] = s sum_n dy[t][n] B[n][j]): one CTA per
// token and 8 ranks.
template <typename TX, bool kGrad>
__global__ void __launch_bounds__(kAdThreads) shrink_kernel(AdParams p)
{
    __shared__ float red[kAdThreads / 32][8];
    const int t = blockIdx.x, j0 = blockIdx.y * 8, tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int a = adapter_at(p, t);
    const int rank = a < 0 ? 0 : rank_of(p, a);
    float acc[8] = {};
    if (j0 < rank) {
        if (kGrad) {
            const TX *dy = static_cast<const TX *>(p.dy) + t * p.lddy;
            const TX *B = static_cast<const TX *>(p.b) + (size_t)a * p.N * p.R;
            for (int n = tid; n < p.N; n += kAdThreads) {
                float f[8];
                to_f32(load8(B + (size_t)n * p.R + j0), f);
                const float d = f32_of(dy[n]);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(d, f[i], acc[i]);
            }
        } else {
            const TX *x = static_cast<const TX *>(p.x) + t * p.ldx;
            const TX *A = static_cast<const TX *>(p.a) + ((size_t)a * p.R + j0) * p.K;
            for (int k = tid * 8; k < p.K; k += kAdThreads * 8) {
                float f[8], g[8];
                to_f32(load8(x + k), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    to_f32(load8(A + (size_t)i * p.K + k), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i] = fmaf(f[e], g[e], acc[i]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
        if ((tid & 31) == 0) red[tid >> 5][i] = acc[i];
    }
    __syncthreads();
    if (tid < 8) {
        float v = 0.f;
        for (int w = 0; w < kAdThreads / 32; ++w) v += red[w][tid];
        if (kGrad && a >= 0) v *= p.scaling[a];
        p.z[(size_t)t * p.R + j0 + tid] = j0 + tid < rank ? v : 0.f;
    }
}

// y[t][n] = y_in[t][n] + s sum_j z[t][j] B[n][j] (kGrad: dx[t][k] = dx_in[t][k] + sum_j
// dz[t][j] A[j][k]): one thread per element.
template <typename TX, typename TY, bool kGrad>
__global__ void __launch_bounds__(kAdThreads) expand_kernel(AdParams p)
{
    __shared__ float s_z[128];
    const int t = blockIdx.x, tid = threadIdx.x, i = blockIdx.y * kAdThreads + tid;
    pdl_trigger();
    pdl_wait();
    const int a = adapter_at(p, t);
    const int rank = a < 0 ? 0 : rank_of(p, a);
    if (tid < rank) s_z[tid] = p.zr[(size_t)t * p.R + tid];
    __syncthreads();
    const int width = kGrad ? p.K : p.N;
    if (i >= width) return;
    const TY *in = static_cast<const TY *>(p.y_in);
    TY *y = static_cast<TY *>(p.y) + t * p.ldy + i;
    if (in) in += t * p.ldy_in + i;
    if (rank == 0) {
        if (in != y) *y = in ? *in : from_f32<TY>(0.f);
        return;
    }
    float acc = 0.f;
    if (kGrad) {
        const TX *A = static_cast<const TX *>(p.a) + (size_t)a * p.R * p.K + i;
        for (int j = 0; j < rank; ++j) acc = fmaf(s_z[j], f32_of(A[(size_t)j * p.K]), acc);
    } else {
        const TX *B = static_cast<const TX *>(p.b) + ((size_t)a * p.N + i) * p.R;
        for (int j = 0; j < rank; ++j) acc = fmaf(s_z[j], f32_of(B[j]), acc);
        acc *= p.scaling[a];
    }
    *y = from_f32<TY>((in ? f32_of(*in) : 0.f) + acc);
}

// da[a][j][k] = sum_t dz[t][j] x[t][k] (kB: db[a][n][j] = s sum_t z[t][j] dy[t][n]): one CTA per
// adapter, rank and 128 columns, over the batch's tokens in order.
template <typename TX, bool kB>
__global__ void __launch_bounds__(kAdThreads) grad_kernel(AdParams p)
{
    const int c = blockIdx.x * kAdThreads + threadIdx.x, j = blockIdx.y, a = blockIdx.z;
    pdl_trigger();
    pdl_wait();
    const int width = kB ? p.N : p.K;
    if (c >= width) return;
    const int rank = rank_of(p, a);
    const TX *x = static_cast<const TX *>(kB ? p.dy : p.x);
    const long long ld = kB ? p.lddy : p.ldx;
    float acc = 0.f;
    bool any = false;
    if (j < rank)
        for (int t = 0; t < p.T; ++t) {
            if (p.adapter_of[t] != a) continue;
            any = true;
            acc = fmaf(p.zr[(size_t)t * p.R + j], f32_of(x[t * ld + c]), acc);
        }
    if (kB) acc *= p.scaling[a];
    float *out = p.out + (kB ? ((size_t)a * p.N + c) * p.R + j : ((size_t)a * p.R + j) * p.K + c);
    if (!p.accumulate) *out = any ? acc : 0.f;
    else if (any) *out += acc;
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype >= MOE_DTYPE_F16 && dtype <= MOE_DTYPE_F32; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

struct AdWs {
    size_t z, total;
};

AdWs ad_layout(const moe_adapters_desc &d, int T)
{
    AdWs w;
    size_t o = 0;
    w.z = o; o = up256(o + (size_t)T * d.max_rank * 4);
    w.total = std::max<size_t>(o, 256);
    return w;
}

bool ld_ok(int64_t ld, int width) { return ld >= width && (uint64_t)ld < (1ull << 40); }

// rows of 16-bit elements that 16-byte loads can read
bool rows16_ok(const void *p, int64_t ld, int width) { return p && aligned16(p) && ld_ok(ld, width) && ld % 8 == 0; }

// rows that the kernels read and write element by element or wider as they are aligned
bool out_ok(const void *p, int dtype, int64_t ld, int width)
{
    return p && known_dtype(dtype) && ld_ok(ld, width) && reinterpret_cast<uintptr_t>(p) % dtype_bytes(dtype) == 0;
}

bool ready(const moe_adapters *h, int T)
{
    int dev = -1;
    return h && T >= 0 && T <= h->desc.max_tokens && cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

int check_ws(const moe_adapters *h, int T, const void *ws, size_t bytes)
{
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || bytes < ad_layout(h->desc, T).total)
        return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

AdParams ad_params(const moe_adapters *h, const int32_t *adapter_of, int T)
{
    AdParams p = {};
    p.a = h->w.a;
    p.b = h->w.b;
    p.scaling = h->w.scaling;
    p.rank = h->w.rank;
    p.adapter_of = adapter_of;
    p.T = T;
    p.K = h->desc.in_features;
    p.N = h->desc.out_features;
    p.R = h->desc.max_rank;
    p.n = h->desc.n_adapters;
    p.status = h->d_status;
    return p;
}

template <typename TX, bool kGrad>
cudaError_t run_expand(const AdParams &p, int y_dtype, cudaStream_t s)
{
    const dim3 grid(p.T, ((kGrad ? p.K : p.N) + kAdThreads - 1) / kAdThreads);
    switch (y_dtype) {
    case MOE_DTYPE_F16: return launch_chained(expand_kernel<TX, __half, kGrad>, grid, kAdThreads, 0, s, p);
    case MOE_DTYPE_BF16: return launch_chained(expand_kernel<TX, __nv_bfloat16, kGrad>, grid, kAdThreads, 0, s, p);
    default: return launch_chained(expand_kernel<TX, float, kGrad>, grid, kAdThreads, 0, s, p);
    }
}

template <typename TX>
cudaError_t run_apply(const AdParams &p, int y_dtype, cudaStream_t s)
{
    const cudaError_t e = launch_chained(shrink_kernel<TX, false>, dim3(p.T, p.R / 8), kAdThreads, 0, s, p);
    return e != cudaSuccess ? e : run_expand<TX, false>(p, y_dtype, s);
}

template <typename TX>
cudaError_t run_backward(AdParams p, const float *z, int dx_dtype, float *da, float *db, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (p.T) e = launch_chained(shrink_kernel<TX, true>, dim3(p.T, p.R / 8), kAdThreads, 0, s, p);
    if (e == cudaSuccess && p.T && p.y) e = run_expand<TX, true>(p, dx_dtype, s);
    if (e != cudaSuccess || !da) return e;
    p.out = da;
    e = launch_chained(grad_kernel<TX, false>, dim3((p.K + kAdThreads - 1) / kAdThreads, p.R, p.n), kAdThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    p.out = db;
    p.zr = z;
    return launch_chained(grad_kernel<TX, true>, dim3((p.N + kAdThreads - 1) / kAdThreads, p.R, p.n), kAdThreads, 0, s,
                          p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_adapters_create(const moe_adapters_desc *desc, const moe_adapters_weights *weights, moe_adapters **out)
{
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    if (!desc || !weights) return MOE_ERR_INVALID_ARG;
    const moe_adapters_desc &d = *desc;
    if (d.in_features < 8 || d.in_features > 16384 || d.in_features % 8) return MOE_ERR_INVALID_ARG;
    if (d.out_features < 1 || d.out_features > 16384) return MOE_ERR_INVALID_ARG;
    if (d.n_adapters < 1 || d.n_adapters > 1024) return MOE_ERR_INVALID_ARG;
    if (d.max_rank < 8 || d.max_rank > 128 || d.max_rank % 8) return MOE_ERR_INVALID_ARG;
    if (d.dtype != MOE_DTYPE_F16 && d.dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
    if (d.max_tokens < 1 || d.max_tokens > 65536) return MOE_ERR_INVALID_ARG;
    const moe_adapters_weights &w = *weights;
    if (!w.a || !w.b || !w.scaling || !aligned16(w.a) || !aligned16(w.b) || !aligned16(w.scaling) ||
        !aligned16(w.rank))
        return MOE_ERR_INVALID_ARG;
    moe_adapters *h = new (std::nothrow) moe_adapters();
    if (!h) return MOE_ERR_CUDA;
    h->desc = d;
    h->w = w;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        cudaMalloc(&h->d_status, 256) != cudaSuccess) {
        delete h;
        return MOE_ERR_CUDA;
    }
    if (cudaMemset(h->d_status, 0, 256) != cudaSuccess) {
        cudaFree(h->d_status);
        delete h;
        return MOE_ERR_CUDA;
    }
    *out = h;
    return MOE_OK;
}

int moe_adapters_destroy(moe_adapters *h)
{
    if (!h) return MOE_OK;
    cudaFree(h->d_status);
    delete h;
    return MOE_OK;
}

size_t moe_adapters_workspace_size(const moe_adapters *h, int T)
{
    if (!h || T < 0 || T > h->desc.max_tokens) return 0;
    return ad_layout(h->desc, T).total;
}

int moe_adapters_apply(const moe_adapters *h, const void *x, int64_t ldx, const int32_t *adapter_of, int T,
                       const void *y_in, int64_t ldy_in, void *y, int y_dtype, int64_t ldy, float *z, void *ws,
                       size_t ws_bytes, moe_stream_t stream)
{
    if (!ready(h, T)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const moe_adapters_desc &d = h->desc;
    if (!rows16_ok(x, ldx, d.in_features) || !adapter_of || !out_ok(y, y_dtype, ldy, d.out_features) ||
        (y_in && !out_ok(y_in, y_dtype, ldy_in, d.out_features)) || (y_in == y && ldy_in != ldy) || !aligned16(z))
        return MOE_ERR_INVALID_ARG;
    const int rc = check_ws(h, T, ws, ws_bytes);
    if (rc) return rc;
    AdParams p = ad_params(h, adapter_of, T);
    p.x = x;
    p.ldx = ldx;
    p.y_in = y_in;
    p.ldy_in = ldy_in;
    p.y = y;
    p.ldy = ldy;
    p.z = z ? z : reinterpret_cast<float *>(static_cast<char *>(ws) + ad_layout(d, T).z);
    p.zr = p.z;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(d.dtype == MOE_DTYPE_F16 ? run_apply<__half>(p, y_dtype, s)
                                                : run_apply<__nv_bfloat16>(p, y_dtype, s));
}

int moe_adapters_backward(const moe_adapters *h, const void *x, int64_t ldx, const float *z, const void *dy,
                          int64_t lddy, const int32_t *adapter_of, int T, const void *dx_in, int64_t lddx_in, void *dx,
                          int dx_dtype, int64_t lddx, float *da, float *db, int accumulate, void *ws, size_t ws_bytes,
                          moe_stream_t stream)
{
    if (!ready(h, T) || !da != !db || !aligned16(da) || !aligned16(db)) return MOE_ERR_INVALID_ARG;
    const moe_adapters_desc &d = h->desc;
    if (d.out_features % 8) return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (!rows16_ok(dy, lddy, d.out_features) || !adapter_of) return MOE_ERR_INVALID_ARG;
        if (da && (!rows16_ok(x, ldx, d.in_features) || !z || !aligned16(z))) return MOE_ERR_INVALID_ARG;
        if (dx && (!out_ok(dx, dx_dtype, lddx, d.in_features) ||
                   (dx_in && !out_ok(dx_in, dx_dtype, lddx_in, d.in_features)) || (dx_in == dx && lddx_in != lddx)))
            return MOE_ERR_INVALID_ARG;
    }
    if (!dx && dx_in) return MOE_ERR_INVALID_ARG;
    if ((T == 0 && (!da || accumulate)) || (!dx && !da)) return MOE_OK;
    const int rc = check_ws(h, T, ws, ws_bytes);
    if (rc) return rc;
    AdParams p = ad_params(h, adapter_of, T);
    p.x = x;
    p.ldx = ldx;
    p.dy = dy;
    p.lddy = lddy;
    p.y_in = dx_in;
    p.ldy_in = lddx_in;
    p.y = dx;
    p.ldy = lddx;
    p.accumulate = accumulate != 0;
    p.z = reinterpret_cast<float *>(static_cast<char *>(ws) + ad_layout(d, T).z);
    p.zr = p.z;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(d.dtype == MOE_DTYPE_F16 ? run_backward<__half>(p, z, dx_dtype, da, db, s)
                                                : run_backward<__nv_bfloat16>(p, z, dx_dtype, da, db, s));
}

int moe_adapters_get_device_status(const moe_adapters *h, int *status)
{
    if (!h || !status) return MOE_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, h->d_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaMemset(h->d_status, 0, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
    *status = v;
    return MOE_OK;
}

}  // extern "C"

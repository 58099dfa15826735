// moe_sort.cu -- tokens sorted by expert and back: the sort itself, the rows' way out
// (dispatch), their weighted way back, and the gradients of both.
#include "moe_internal.h"
#include "moe_rows.cuh"
#include "moe_tcgen05.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;   // chunks of a cluster
constexpr int kRowThreads = 256;

// the bin of a key, or -1 for an entry that is dropped; other keys than -1 that lie
// outside [0, bins) are an error of the caller
__device__ __forceinline__ int bin_of(int key, int bins, int none_bin, int *status)
{
    if (key >= 0 && key < bins) return key;
    if (key != -1) record_error(status, MOE_ERR_DEVICE_BOUNDS);
    return none_bin;
}

// keys that name a bin directly: with a none_bin (the last one) the others
__device__ __forceinline__ int key_bins(const SortParams &p) { return p.none_bin >= 0 ? p.E - 1 : p.E; }

// Exclusive scan of v[0 .. E) in place over the whole block; v[E] receives the sum.
__device__ void block_scan(int *v, int E, int *warp_sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (E + kSortThreads - 1) / kSortThreads;
    const int lo = min(tid * per, E), hi = min(lo + per, E);
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += v[i];
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += warp_sums[w];
    for (int i = lo; i < hi; ++i) {
        const int t = v[i];
        v[i] = run;
        run += t;
    }
    if (tid == kSortThreads - 1) v[E] = run;   // (the last thread's run ends at the total)
    __syncthreads();
}

// Histogram of each chunk of kSortChunk keys (more chunks than a cluster holds).
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(SortParams p)
{
    extern __shared__ int s_hist[];
    pdl_trigger();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) s_hist[e] = 0;
    pdl_wait();
    __syncthreads();
    const int base = blockIdx.x * kSortChunk, end = min(base + kSortChunk, p.n);
#pragma unroll 8
    for (int i = base + threadIdx.x; i < end; i += kSortThreads) {
        const int e = bin_of(__ldcg(p.key + i), key_bins(p), p.none_bin, nullptr);
        if (e >= 0) atomicAdd(s_hist + e, 1);   // (integer counts: any order gives the same)
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) p.hist[(size_t)blockIdx.x * p.E + e] = s_hist[e];
}

// Positions of one chunk's entries: a warp owns 256 consecutive entries and ranks them 32
// at a time (match_any: entries of equal key in lane order), which keeps the sort stable;
// the chunks before give each bin's base.  Up to 8 chunks (16384 entries) are one cluster,
// whose CTAs read one another's counts from shared memory; more take them from
// sort_hist_kernel.  Work is O(n + chunks * E); for the layer's batches it is latency: one
// pass over the keys, a scan of E counts, one write.
template <bool kCluster>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortParams p)
{
    extern __shared__ int sm[];
    int *seg = sm;                         // [E + 1]
    int *base = seg + p.E + 1;             // [E] entries of the bin in the chunks before
    int *all = base + p.E;                 // [E] entries of the bin
    int *own = all + p.E;                  // [E] entries of the bin in this chunk
    uint16_t *wh = reinterpret_cast<uint16_t *>(own + p.E);   // [kSortWarps][E]: entries of each bin per warp
    __shared__ int warp_sums[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = blockIdx.x, chunks = gridDim.x;
    pdl_trigger();
    for (int i = tid; i < kSortWarps * p.E; i += kSortThreads) wh[i] = 0;
    pdl_wait();
    __syncthreads();

    constexpr int kIter = kSortChunk / kSortThreads;   // 8 rounds of 32 entries per warp
    const int first = chunk * kSortChunk + warp * (kIter * 32) + lane;
    int bin[kIter], rank[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {   // (all the loads first: recording a bad key would order them)
        const int i = first + it * 32;
        bin[it] = i < p.n ? __ldcg(p.key + i) : -1;
    }
#pragma unroll
    for (int it = 0; it < kIter; ++it)
        bin[it] = first + it * 32 < p.n ? bin_of(bin[it], key_bins(p), p.none_bin, p.status) : -1;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const unsigned same = __match_any_sync(0xffffffffu, bin[it]);
        int before = 0;
        if (bin[it] >= 0) before = wh[warp * p.E + bin[it]];
        __syncwarp();
        if (bin[it] >= 0 && (same & ((1u << lane) - 1u)) == 0u) wh[warp * p.E + bin[it]] = static_cast<uint16_t>(before + __popc(same));
        __syncwarp();
        rank[it] = before + __popc(same & ((1u << lane) - 1u));
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += kSortThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = wh[w * p.E + e];
            wh[w * p.E + e] = static_cast<uint16_t>(run);
            run += c;
        }
        own[e] = run;
    }
    if (kCluster) cluster_sync();   // (a thread reads its own bins: no barrier without peers)
    for (int e = tid; e < p.E; e += kSortThreads) {
        int before = 0, total = 0;
        if (kCluster) {
            int part[kSortCluster];
#pragma unroll
            for (int c = 0; c < kSortCluster; ++c)
                part[c] = c < chunks ? __float_as_int(ld_cluster(peer_addr(smem_u32(own + e), c))) : 0;
#pragma unroll
            for (int c = 0; c < kSortCluster; ++c) {
                before += c < chunk ? part[c] : 0;
                total += part[c];
            }
        } else if (chunks > 1) {
#pragma unroll 4
            for (int c = 0; c < chunks; ++c) {
                const int h = __ldcg(p.hist + (size_t)c * p.E + e);
                before += c < chunk ? h : 0;
                total += h;
            }
        } else {
            total = own[e];
        }
        base[e] = before;
        all[e] = total;
        seg[e] = (total + p.align - 1) / p.align * p.align;
        if (chunk == 0 && p.counts) p.counts[e] = total;
    }
    __syncthreads();
    block_scan(seg, p.E, warp_sums);
    if (chunk == 0)
        for (int e = tid; e <= p.E; e += kSortThreads) p.seg[e] = seg[e];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int i = first + it * 32;
        if (i >= p.n) continue;
        const int e = bin[it];
        const int pos = e < 0 ? -1 : seg[e] + base[e] + wh[warp * p.E + e] + rank[it];
        if (p.row_of) p.row_of[i] = pos;
        if (p.entry_of && pos >= 0) p.entry_of[pos] = i;
    }
    if (chunk == 0) {
        for (int i = tid; i < p.n_zero; i += kSortThreads) p.zero[i] = 0u;
        if (p.order && tid < p.E - 1) {
            int at = 0;
            for (int e = 0; e < p.E - 1; ++e) at += all[e] > all[tid] || (all[e] == all[tid] && e < tid);
            p.order[at] = tid;
        }
        if (p.tile_bin) {
            for (int e = tid; e < p.E; e += kSortThreads)
                for (int i = seg[e] / p.align; i < seg[e + 1] / p.align; ++i) p.tile_bin[i] = e;
            for (int i = seg[p.E] / p.align + tid; i < p.max_tiles; i += kSortThreads) p.tile_bin[i] = -1;
        }
    }
    // the padding behind each group's entries
    if (p.entry_of && chunk == 0)
        for (int e = warp; e < p.E; e += kSortWarps)
            for (int pos = seg[e] + all[e] + lane; pos < seg[e + 1]; pos += 32) p.entry_of[pos] = -1;
    if (kCluster) cluster_sync();   // no CTA leaves while a peer reads its counts
}

// ---------------------------------------------------------------------------- rows out
// rows[row_of[t, j]] = x[t]: x is read once and written k times, so the kernel is bound by
// the writes.  A CTA owns a slice of one token's row; blocks past the last token zero the
// padding rows behind one expert's rows.
struct CopyParams {
    const uint4 *x;
    uint4 *rows;
    long long ldx;        // 16-byte units between rows of x
    int row16;            // 16-byte units of a row
    int T, k, E;
    const int32_t *row_of, *counts, *seg;
};

// one CTA's slice of token t's row to the rows s_row[0 .. k)
__device__ __forceinline__ void copy_token(const CopyParams &p, int t, const int *s_row)
{
    const int stride = gridDim.y * kRowThreads, i0 = blockIdx.y * kRowThreads + threadIdx.x;
    const uint4 *src = p.x + (size_t)t * p.ldx;
    constexpr int kU = 4;
    for (int b = i0; b < p.row16; b += kU * stride) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (b + u * stride < p.row16) v[u] = src[b + u * stride];
        for (int j = 0; j < p.k; ++j) {
            const int r = s_row[j];
            if (r < 0) continue;
            uint4 *dst = p.rows + (size_t)r * p.row16 + b;
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (b + u * stride < p.row16) dst[u * stride] = v[u];
        }
    }
}

// one CTA's slice of the padding rows [lo, hi)
__device__ __forceinline__ void zero_rows(const CopyParams &p, int lo, int hi)
{
    const int stride = gridDim.y * kRowThreads, i0 = blockIdx.y * kRowThreads + threadIdx.x;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (int r = lo; r < hi; ++r)
        for (int i = i0; i < p.row16; i += stride) p.rows[(size_t)r * p.row16 + i] = z;
}

__global__ void __launch_bounds__(kRowThreads) sort_copy_kernel(CopyParams p)
{
    __shared__ int s_row[kMaxTopK];
    const int tid = threadIdx.x, t = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    if (t >= p.T) {
        const int e = t - p.T;
        zero_rows(p, p.seg[e] + p.counts[e], p.seg[e + 1]);
        return;
    }
    if (tid < p.k) s_row[tid] = p.row_of[(size_t)t * p.k + tid];
    __syncthreads();
    copy_token(p, t, s_row);
}

// The sort and the copy of a decode-sized batch (at most kSmallSort assignments) in one
// launch: every CTA counts all the keys itself (a few per thread), scans the counts and ranks
// its own token's assignments, so that nothing waits for another CTA.  Rows of 6144 bf16, 8 of
// 256 experts, a call in a graph: 256 assignments 3.7 us (two launches 5.5), 1024 6.3 (8.0),
// 2048 13.4 (12.7).
constexpr int kSmallSort = 1024;

__global__ void __launch_bounds__(kRowThreads) sort_small_kernel(SortParams s, CopyParams p)
{
    extern __shared__ int sm[];
    int *key = sm;                 // [n] bins
    int *cnt = key + s.n;          // [E]
    int *seg = cnt + s.E;          // [E + 1]
    __shared__ int warp_sums[kSortWarps];
    __shared__ int s_row[kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = blockIdx.x;
    const bool first = t == 0 && blockIdx.y == 0;
    pdl_trigger();
    for (int e = tid; e < s.E; e += kRowThreads) cnt[e] = 0;
    pdl_wait();
    __syncthreads();
    for (int i = tid; i < s.n; i += kRowThreads) {
        const int e = bin_of(s.key[i], s.E, -1, first ? s.status : nullptr);
        key[i] = e;
        if (e >= 0) atomicAdd(cnt + e, 1);
    }
    __syncthreads();
    for (int e = tid; e < s.E; e += kRowThreads) seg[e] = (cnt[e] + s.align - 1) / s.align * s.align;
    __syncthreads();
    block_scan(seg, s.E, warp_sums);
    if (first)
        for (int e = tid; e <= s.E; e += kRowThreads) {
            s.seg[e] = seg[e];
            if (e < s.E) s.counts[e] = cnt[e];
        }
    if (t >= p.T) {
        const int e = t - p.T;
        zero_rows(p, seg[e] + cnt[e], seg[e + 1]);
        return;
    }
    for (int j = warp; j < p.k; j += kSortWarps) {   // the assignments before mine that share my expert
        const int a = t * p.k + j, e = key[a];
        int before = 0;
        for (int i = lane; i < a; i += 32) before += key[i] == e;
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            s_row[j] = e < 0 ? -1 : seg[e] + before;
            if (blockIdx.y == 0) s.row_of[a] = s_row[j];
        }
    }
    __syncthreads();
    copy_token(p, t, s_row);
}

// ---------------------------------------------------------------------------- rows back
// y[t] = shared[t] + sum_j w[t, j] rows[row_of[t, j]], summed in fp32 in that order and
// rounded once (w = NULL: weights 1, the gradient of the way out).  Reads k rows per
// token and writes one: bound by the reads.  A thread owns 8 elements of the row and keeps
// up to 8 rows' loads in flight.
struct UnsortParams {
    const void *rows;
    const float *w, *shared;
    void *y;
    long long ldy;
    const int32_t *row_of;
    int T, k, H, n_rows;
    int *status;
};

template <typename TR, typename TY>
__global__ void __launch_bounds__(kRowThreads) unsort_kernel(UnsortParams p)
{
    __shared__ int s_row[kMaxTopK];
    __shared__ float s_w[kMaxTopK];
    __shared__ int s_n;
    const int tid = threadIdx.x, t = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    if (tid < 32) {   // the live entries of the token, in j order
        int r = -1;
        float w = 1.f;
        if (tid < p.k) {
            r = p.row_of[(size_t)t * p.k + tid];
            if (p.w) w = p.w[(size_t)t * p.k + tid];
            if (r < -1 || r >= p.n_rows) {
                record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
                r = -1;
            }
            if (w == 0.f) r = -1;
        }
        const unsigned live = __ballot_sync(0xffffffffu, r >= 0);
        if (r >= 0) {
            const int at = __popc(live & ((1u << tid) - 1u));
            s_row[at] = r;
            s_w[at] = w;
        }
        if (tid == 0) s_n = __popc(live);
    }
    __syncthreads();
    const int n = s_n;
    const TR *rows = static_cast<const TR *>(p.rows);
    TY *y = static_cast<TY *>(p.y) + (size_t)t * p.ldy;
    const int stride = gridDim.y * kRowThreads * 8;
    for (int h = (blockIdx.y * kRowThreads + tid) * 8; h < p.H; h += stride) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (p.shared) to_f32(load8(p.shared + (size_t)t * p.H + h), acc);
        constexpr int kU = sizeof(TR) == 2 ? 8 : 4;
        for (int j = 0; j < n; j += kU) {
            Vec8<TR> v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (j + u < n) v[u] = load8(rows + (size_t)s_row[j + u] * p.H + h);
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (j + u < n) {
                    float f[8];
                    to_f32(v[u], f);
                    const float w = s_w[j + u];
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
                }
        }
        store8(y + h, pack8<TY>(acc));
    }
}

// ---------------------------------------------------------------------------- their gradient
// drows[row_of[a]] = w[a] dy[t], dw[a] = <dy[t], rows[row_of[a]]>: reads and writes one row
// per assignment (dy comes from L1 or L2 after its first use), bound by that traffic.
// kWarps warps share an assignment's row; their partial dot products are added in warp
// order.  Blocks past the last assignment zero one expert's padding rows.
struct UnsortGradParams {
    const void *dy, *rows;
    void *drows;
    const float *w;
    float *dw;
    long long lddy;
    const int32_t *row_of, *counts, *seg;
    int T, k, H, E, n_rows, n_blocks;
    int *status;
};

template <typename TR, typename TD, int kWarps>
__global__ void __launch_bounds__(kRowThreads) unsort_grad_kernel(UnsortGradParams p)
{
    constexpr int kPer = kRowThreads / 32 / kWarps;   // assignments per CTA
    __shared__ float s_dot[kRowThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    TR *drows = static_cast<TR *>(p.drows);
    if ((int)blockIdx.x >= p.n_blocks) {
        const int e = blockIdx.x - p.n_blocks;
        const int seg = p.seg[e], lo = seg + p.counts[e], hi = p.seg[e + 1];
        if (seg < 0 || lo < seg || hi > p.n_rows) {
            if (tid == 0) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
            return;
        }
        const Vec8<TR> z = {};
        for (int r = lo; r < hi; ++r)
            for (int h = tid * 8; h < p.H; h += kRowThreads * 8) store8(drows + (size_t)r * p.H + h, z);
        return;
    }
    const size_t a = (size_t)blockIdx.x * kPer + warp / kWarps;
    const int part = warp % kWarps;
    const bool live_a = a < (size_t)p.T * p.k;
    int r = -1;
    float w = 0.f;
    if (live_a) {
        r = p.row_of[a];
        w = p.w[a];
        if (r < -1 || r >= p.n_rows) {
            if (lane == 0) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
            r = -1;
        }
    }
    float dots[8] = {};   // (apart, so that no sum is a long chain)
    if (r >= 0) {
        const TD *dy = static_cast<const TD *>(p.dy) + (a / p.k) * p.lddy;
        const TR *row = static_cast<const TR *>(p.rows) + (size_t)r * p.H;
        TR *drow = drows + (size_t)r * p.H;
        constexpr int kU = 4;
        constexpr int step = kWarps * 32 * 8;
        for (int b = (part * 32 + lane) * 8; b < p.H; b += kU * step) {
            Vec8<TR> v[kU];
            Vec8<TD> d[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (b + u * step < p.H) {
                    v[u] = load8(row + b + u * step);
                    d[u] = load8(dy + b + u * step);
                }
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (b + u * step < p.H) {
                    float f[8], g[8];
                    to_f32(v[u], f);
                    to_f32(d[u], g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dots[i] = fmaf(f[i], g[i], dots[i]);
                        g[i] = w == 0.f ? 0.f : w * g[i];   // weight 0: the forward pass skipped the row
                    }
                    store8(drow + b + u * step, pack8<TR>(g));
                }
        }
    }
    float dot = ((dots[0] + dots[1]) + (dots[2] + dots[3])) + ((dots[4] + dots[5]) + (dots[6] + dots[7]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (kWarps > 1) {
        if (lane == 0) s_dot[warp] = dot;
        __syncthreads();
        dot = 0.f;
        for (int i = 0; i < kWarps; ++i) dot += s_dot[warp - part + i];
    }
    if (live_a && part == 0 && lane == 0) p.dw[a] = dot;
}

// slices of a row so that `units` rows fill the machine about twice over
int row_slices(int units, int row_steps, int num_sms)
{
    const int want = (2 * num_sms + units - 1) / std::max(units, 1);
    return std::max(1, std::min(want, row_steps));
}

template <typename F>
cudaError_t by_type(int dtype, F &&f)
{
    switch (dtype) {
    case MOE_DTYPE_F16: return f(__half());
    case MOE_DTYPE_BF16: return f(__nv_bfloat16());
    default: return f(float());
    }
}

}  // namespace

cudaError_t launch_sort(const SortParams &p, cudaStream_t s)
{
    const int chunks = std::max(1, (p.n + kSortChunk - 1) / kSortChunk);
    const size_t smem = (size_t)(4 * p.E + 1) * 4 + (size_t)kSortWarps * p.E * 2;   // 32,804 bytes at most (1025 bins)
    if (chunks > 1 && chunks <= kSortCluster)
        return launch_chained(sort_place_kernel<true>, {dim3(chunks), kSortThreads, smem, chunks, s}, p);
    if (chunks > 1) {
        const cudaError_t e = launch_chained(sort_hist_kernel, {dim3(chunks), kSortThreads, (size_t)p.E * 4, 1, s}, p);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(sort_place_kernel<false>, {dim3(chunks), kSortThreads, smem, 1, s}, p);
}

// the sort of `s` and the copy of its rows
cudaError_t launch_sort_rows(const SortParams &s, const void *x, size_t ldx_bytes, size_t row_bytes, int T, int k,
                             void *rows, int num_sms, cudaStream_t stream)
{
    CopyParams p = {};
    p.x = static_cast<const uint4 *>(x);
    p.rows = static_cast<uint4 *>(rows);
    p.ldx = (long long)(ldx_bytes / 16);
    p.row16 = (int)(row_bytes / 16);
    p.T = T;
    p.k = k;
    p.E = s.E;
    p.row_of = s.row_of;
    p.counts = s.counts;
    p.seg = s.seg;
    const int slices = row_slices(T, (p.row16 + kRowThreads - 1) / kRowThreads, num_sms);
    ChainLaunch l = {dim3(T + (s.align > 1 ? s.E : 0), slices), kRowThreads, 0, 1, stream};
    if (T > 0 && s.n <= kSmallSort) {
        l.smem = (size_t)(s.n + 2 * s.E + 1) * 4;
        return launch_chained(sort_small_kernel, l, s, p);
    }
    const cudaError_t e = launch_sort(s, stream);
    return e != cudaSuccess || T == 0 ? e : launch_chained(sort_copy_kernel, l, p);
}

cudaError_t launch_unsort(const void *rows, int rows_dtype, int n_rows, const int32_t *row_of, const float *w, int T,
                          int k, int H, const float *shared, void *y, int y_dtype, long long ldy, int *status,
                          int num_sms, cudaStream_t s)
{
    UnsortParams p = {rows, w, shared, y, ldy, row_of, T, k, H, n_rows, status};
    const int slices = row_slices(T, (H / 8 + kRowThreads - 1) / kRowThreads, num_sms);
    return by_type(rows_dtype, [&](auto tr) {
        return by_type(y_dtype, [&](auto ty) {
            return launch_chained(unsort_kernel<decltype(tr), decltype(ty)>, {dim3(T, slices), kRowThreads, 0, 1, s}, p);
        });
    });
}

cudaError_t launch_unsort_grad(const void *dy, int dy_dtype, long long lddy, const void *rows, int rows_dtype,
                               int n_rows, const int32_t *row_of, const float *w, const int32_t *counts,
                               const int32_t *seg, int T, int k, int H, int E, void *drows, float *dw, int *status,
                               int num_sms, cudaStream_t s)
{
    UnsortGradParams p = {};
    p.dy = dy;
    p.rows = rows;
    p.drows = drows;
    p.w = w;
    p.dw = dw;
    p.lddy = lddy;
    p.row_of = row_of;
    p.counts = counts;
    p.seg = seg;
    p.T = T;
    p.k = k;
    p.H = H;
    p.E = E;
    p.n_rows = n_rows;
    p.status = status;
    const int n = T * k;
    // a CTA per assignment while warps would leave SMs idle (rows of 6144 bf16: 296 assignments
    // 2.6 us against 6.1, 2048 12.3 against 12.1, 3200 18.0 against 15.3)
    const bool few = n < 8 * 2 * num_sms;
    p.n_blocks = few ? n : (n + kRowThreads / 32 - 1) / (kRowThreads / 32);
    const ChainLaunch l = {dim3(p.n_blocks + (seg ? E : 0)), kRowThreads, 0, 1, s};
    return by_type(rows_dtype, [&](auto tr) {
        return by_type(dy_dtype, [&](auto td) {
            using R = decltype(tr);
            using D = decltype(td);
            return few ? launch_chained(unsort_grad_kernel<R, D, kRowThreads / 32>, l, p)
                       : launch_chained(unsort_grad_kernel<R, D, 1>, l, p);
        });
    });
}

}  // namespace moe

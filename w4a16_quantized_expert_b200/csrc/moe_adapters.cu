// moe_adapters.cu -- low-rank adapters of many requests beside a shared projection, and
// their gradients: kernels and entry points.
//
// y = y_in + s B (A x) per token is two thin products: the shrink z = A x contracts the long
// axis and the expand adds s B z over it.  Both are bound by the rows of x and y (or, for a
// few tokens, by the adapters' weights and launch latency) as long as the products run on
// the tensor cores.  Batches of at most 32 tokens take two latency-sized kernels
// (shrink_few_kernel, expand_few_kernel); larger ones are sorted by adapter into tiles of
// 128 tokens and take the tcgen05 kernels (shrink_tile_kernel, expand_tile_kernel,
// grad_tile_kernel), and so does every gradient.
//
// z enters a second product, whose operands are 16-bit.  It is carried as a sum of pieces,
// each the rounding of what the ones before leave: two in fp16 (22 bits), under a power of
// two per row (the gradient of the weights: per adapter) that keeps them in fp16's range;
// three in bf16 (all 24 bits).  The products' error stays at fp32's level, where a single
// rounding of z to 16 bits would cost up to 2^-9 of the result and two bf16 pieces 3e-6
// (measured on weight gradients, against 8e-7 for the same sums in fp32).
#include "moe_internal.h"
#include "moe_rows.cuh"
#include "moe_tcgen05.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <new>
#include <type_traits>

// the opaque handle
struct moe_adapters {
    moe_adapters_desc desc;
    moe_adapters_weights w;
    // boxes of 64 columns: A [ranks], B [128 rows], B [64 rows]
    CUtensorMap map_a, map_b, map_b64;
    int *d_status;
    int device;
    int num_sms;
};

namespace moe {
namespace {

// Tokens of the latency-sized path (one warp plans the batch).  At 32 tokens of 6144 x 6144 it
// takes 9.6 us with 32 adapters of rank 16 where the tiles take 31, 21 against 34 at rank 64,
// 14 against 17 with one adapter of rank 64.
constexpr int kFewT = 32;
constexpr int kFewThreads = 128;
constexpr int kFewK = 256;         // K values per CTA of the small shrink
constexpr int kFewN = 128;         // columns per CTA of the small expand
constexpr int kTile = 128;         // tokens per tile of the tcgen05 kernels (MMA M)
constexpr int kBlk = kTile * 128;  // bytes of a [128 rows][64 columns] 16-bit block
constexpr int kWorkers = 256;      // load and epilogue threads of a tcgen05 CTA
constexpr int kTcThreads = kWorkers + 32;   // and its MMA warp
constexpr int kMmaWarp = kWorkers / 32, kTmaWarp = kMmaWarp + 1;
constexpr size_t kMaxSmem = 224 * 1024;     // of a ring
constexpr int kOrdered = 128;      // adapters that the sort ranks by size
constexpr int kMaxSplit = 8;       // CTAs of a cluster that share a contraction

struct AdParams {
    const void *x, *dy;          // [T][K], [T][N] of the pool's type
    const void *a, *b;
    const float *scaling;
    const int32_t *rank, *adapter_of;
    const void *y_in;
    void *y;                     // y, or dx
    const float *z_in;           // z of the forward call (gradient)
    float *z_out;                // optional z of this call
    float *da, *db;
    long long ldx, lddy, ldy_in, ldy;
    int T, K, N, R, Kp, n, accumulate, want_dw;
    // the plan: tokens sorted by adapter, tiles of 128 positions
    int32_t *seg, *counts, *entry_of, *tile_bin;
    int32_t *order;              // adapters, most tokens first (NULL: as they are numbered)
    // intermediates, by position: z (dz) as pieces [kPieces][Kp], the scale that undoes theirs
    void *pieces, *zl, *dl;
    float *row_scale, *dz;
    unsigned *amax;              // [2][n] largest |dz|, |z| of each adapter (fp16 pools)
    float *z_part;               // small path: [splits][T][R]
    int splits;
    int *status;
};

__device__ __forceinline__ int rank_of(const AdParams &p, int bin)
{
    if (bin >= p.n) return 0;
    if (!p.rank) return p.R;
    const int r = __ldcg(p.rank + bin);
    if (r >= 0 && r <= p.R) return r;
    record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
    return 0;
}

// the power of two that brings a largest magnitude m into [1, 4), and its inverse
__device__ __forceinline__ float norm_scale(float m, float &inverse)
{
    int e = static_cast<int>((__float_as_uint(m) >> 23) & 0xFFu);
    e = min(max(e, 1), 253);
    inverse = pow2f(e - 127);
    return pow2f(127 - e);
}

__device__ __forceinline__ float finite_or_0(float v) { return fabsf(v) <= 3.4028234663852886e38f ? fabsf(v) : 0.f; }

template <typename T>
constexpr int kPieces = TcType<T>::code ? 3 : 2;

// v as pieces; an infinite or NaN piece stands alone
template <typename T>
__device__ __forceinline__ void split_pieces(float v, T (&piece)[kPieces<T>])
{
#pragma unroll
    for (int i = 0; i < kPieces<T>; ++i) {
        piece[i] = from_f32<T>(v);
        const float h = f32_of(piece[i]);
        v = fabsf(h) <= 3.4028234663852886e38f ? v - h : 0.f;
    }
}

// the same to a row of pieces, `stride` apart
template <typename T>
__device__ __forceinline__ void store_pieces(float v, T *dst, int stride)
{
    T piece[kPieces<T>];
    split_pieces(v, piece);
#pragma unroll
    for (int i = 0; i < kPieces<T>; ++i) dst[i * stride] = piece[i];
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

template <typename T>
__device__ __forceinline__ void mma_t(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1);
template <>
__device__ __forceinline__ void mma_t<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    mma_16816(c, a0, a1, a2, a3, b0, b1);
}
template <>
__device__ __forceinline__ void mma_t<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                     uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ============================================================================ few tokens
// Tile `tile` of a batch of at most 32 tokens: up to 16 tokens of one adapter, in token
// order.  One ballot per warp finds the tiles' first tokens.  Returns the adapter (n: tokens
// without one), or -1 if there is no such tile; s_tok[0 .. cnt) receives the tokens.
__device__ __forceinline__ int few_tile(const AdParams &p, int tile, int *s_tok, int &cnt)
{
    const int lane = threadIdx.x & 31;
    int bin = -1 - lane;   // lanes without a token: alone in their group
    if (lane < p.T) {
        bin = __ldcg(p.adapter_of + lane);
        if (bin < 0 || bin >= p.n) {
            if (bin != -1) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
            bin = p.n;
        }
    }
    const unsigned below = (1u << lane) - 1u;
    const unsigned same = __match_any_sync(0xffffffffu, bin);
    const int at = __popc(same & below);
    const unsigned first = __ballot_sync(0xffffffffu, bin >= 0 && at % 16 == 0);
    const bool mine = bin >= 0 && at % 16 == 0 && __popc(first & below) == tile;
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (!who) return -1;
    const int lead = __ffs(who) - 1;
    const int tile_bin = __shfl_sync(0xffffffffu, bin, lead), at0 = __shfl_sync(0xffffffffu, at, lead);
    const bool in = bin == tile_bin && at >= at0 && at < at0 + 16;
    cnt = __popc(__ballot_sync(0xffffffffu, in));
    if (in && threadIdx.x < 32) s_tok[at - at0] = lane;
    return tile_bin;
}

// z_part[split][t][j] = sum over the split's 256 K of x[t][k] A[j][k].  No shared-memory
// staging: a thread's 16 bytes of a row are its operand of two m16n8k16 steps (the order of
// K inside a product is free as long as both operands agree), so every load is issued up
// front and the kernel is one memory latency long.  CTA (split, tile), 64 K per warp.
template <typename TX, int NB>
__global__ void __launch_bounds__(kFewThreads) shrink_few_kernel(const AdParams p)
{
    __shared__ int s_tok[16];
    __shared__ float red[kFewThreads / 32][16][NB * 8 + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
    pdl_wait();
    pdl_trigger();   // (the expand kernel may now read what earlier grids wrote)
    int cnt = 0;
    const int bin = few_tile(p, blockIdx.y, s_tok, cnt);
    if (bin < 0 || bin == p.n) return;
    __syncthreads();
    const TX *A = static_cast<const TX *>(p.a) + (size_t)bin * p.R * p.K;
    const TX *x0 = static_cast<const TX *>(p.x) + (g < cnt ? s_tok[g] : 0) * p.ldx;
    const TX *x1 = static_cast<const TX *>(p.x) + (g + 8 < cnt ? s_tok[g + 8] : 0) * p.ldx;
    float acc[NB][4] = {};
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int k0 = blockIdx.x * kFewK + warp * 64 + tig * 8;
    constexpr int kU = NB > 8 ? 1 : 2;   // 32-K blocks whose loads are in flight together
#pragma unroll
    for (int b0 = 0; b0 < 2; b0 += kU) {
        uint4 xa[kU], xb[kU], av[kU][NB];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int k = k0 + (b0 + u) * 32;
            const bool in = k < p.K;
            xa[u] = in && g < cnt ? *reinterpret_cast<const uint4 *>(x0 + k) : zero;
            xb[u] = in && g + 8 < cnt ? *reinterpret_cast<const uint4 *>(x1 + k) : zero;
#pragma unroll
            for (int j = 0; j < NB; ++j)
                av[u][j] = in && j * 8 + g < p.R
                               ? *reinterpret_cast<const uint4 *>(A + (size_t)(j * 8 + g) * p.K + k) : zero;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                mma_t<TX>(acc[j], xa[u].x, xb[u].x, xa[u].y, xb[u].y, av[u][j].x, av[u][j].y);
                mma_t<TX>(acc[j], xa[u].z, xb[u].z, xa[u].w, xb[u].w, av[u][j].z, av[u][j].w);
            }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        red[warp][g][j * 8 + 2 * tig] = acc[j][0];
        red[warp][g][j * 8 + 2 * tig + 1] = acc[j][1];
        red[warp][g + 8][j * 8 + 2 * tig] = acc[j][2];
        red[warp][g + 8][j * 8 + 2 * tig + 1] = acc[j][3];
    }
    __syncthreads();
    for (int i = tid; i < cnt * p.R; i += kFewThreads) {
        const int row = i / p.R, j = i % p.R;
        float v = red[0][row][j];
#pragma unroll
        for (int w = 1; w < kFewThreads / 32; ++w) v += red[w][row][j];
        p.z_part[((size_t)blockIdx.x * p.T + s_tok[row]) * p.R + j] = v;
    }
}

// y[t][n] = y_in[t][n] + s sum_j z[t][j] B[n][j] for 128 columns and a tile of up to 16
// tokens.  B and y_in are loaded before the wait for the shrink kernel (which has itself
// seen every earlier grid complete before this one may start), so after it only the
// partial sums of z stand between the launch and the result.
//
// The fp32 output of rank 64 is held to the registers of 5 CTAs per SM, which it would miss by two
// (32 tokens of 6144 x 6144: 24.8 us, 28.2 with 4).
template <typename TX, typename TY, int KB>
__global__ void __launch_bounds__(kFewThreads, KB == 4 && sizeof(TY) == 4 ? 5 : 0) expand_few_kernel(const AdParams p)
{
    constexpr int W = KB * 16;
    __shared__ int s_tok[16];
    __shared__ float s_scale[16], s_z[16][W];
    __shared__ __align__(8) TX s_p[kPieces<TX>][16][W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
    pdl_trigger();
    int cnt = 0;
    const int bin = few_tile(p, blockIdx.y, s_tok, cnt);
    if (bin < 0) {
        pdl_wait();
        return;
    }
    __syncthreads();
    const int rank = rank_of(p, bin);
    const int n0 = blockIdx.x * kFewN + warp * 32;
    const TY *in = static_cast<const TY *>(p.y_in);
    TY *y = static_cast<TY *>(p.y);
    const int rows[2] = {g < cnt ? s_tok[g] : -1, g + 8 < cnt ? s_tok[g + 8] : -1};
    if (rank == 0) {
        pdl_wait();
        if (p.z_out && blockIdx.x == 0)
            for (int i = tid; i < cnt * p.R; i += kFewThreads) p.z_out[(size_t)s_tok[i / p.R] * p.R + i % p.R] = 0.f;
        if (in == y) return;
        for (int r = 0; r < cnt; ++r)   // the base's bits
            if (n0 + lane < p.N)
                y[s_tok[r] * p.ldy + n0 + lane] = in ? in[s_tok[r] * p.ldy_in + n0 + lane] : from_f32<TY>(0.f);
        return;
    }
    const float scaling = __ldcg(p.scaling + bin);
    const TX *B = static_cast<const TX *>(p.b) + (size_t)bin * p.N * p.R;
    uint2 bv[4][KB];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + i * 8 + g;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int j = k * 16 + tig * 4;
            bv[i][k] = make_uint2(0u, 0u);
            if (n < p.N && j < rank) {   // (j < rank <= R: the four values are inside the row)
                bv[i][k] = __ldcg(reinterpret_cast<const uint2 *>(B + (size_t)n * p.R + j));
                if (j + 1 >= rank) bv[i][k].x &= 0xFFFFu;
                if (j + 2 >= rank) bv[i][k].y = 0u;
                else if (j + 3 >= rank) bv[i][k].y &= 0xFFFFu;
            }
        }
    }
    float yv[2][4][2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = n0 + i * 8 + tig * 2 + e;
                yv[r][i][e] = in && rows[r] >= 0 && n < p.N ? f32_of(__ldcg(in + rows[r] * p.ldy_in + n)) : 0.f;
            }
    pdl_wait();
    // z: the splits' sums: a few lanes per value when there are few values, else a thread per
    // four values (32 tokens of one adapter of rank 64: 16.0 -> 14.4 us; two splits in flight:
    // four cost registers, hence CTAs per SM, and 16 adapters of one token 9.1 us for 8.2)
    auto put = [&](int row, int j, float v) {
        v = j < rank ? v : 0.f;
        s_z[row][j] = v;
        if (p.z_out && blockIdx.x == 0) p.z_out[(size_t)s_tok[row] * p.R + j] = v;
    };
    const int n_el = cnt * p.R;
    const size_t split = (size_t)p.T * p.R;
    if (n_el <= 128) {
        const int L = n_el <= 16 ? 8 : n_el <= 32 ? 4 : n_el <= 64 ? 2 : 1, part = tid % L, e = tid / L;
        const int row = min(e, n_el - 1) / p.R, j = min(e, n_el - 1) % p.R;
        const float *src = p.z_part + (size_t)s_tok[row] * p.R + j;
        float v = 0.f;
#pragma unroll 8
        for (int s = part; s < p.splits; s += L) v += __ldcg(src + s * split);
        for (int off = L >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (e < n_el && part == 0) put(row, j, v);
    } else {
        for (int e = tid * 4; e < n_el; e += kFewThreads * 4) {
            const int row = e / p.R, j = e % p.R;
            const float *src = p.z_part + (size_t)s_tok[row] * p.R + j;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int s = 0; s < p.splits; ++s) {
                const float4 o = __ldcg(reinterpret_cast<const float4 *>(src + s * split));
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            put(row, j, v.x);
            put(row, j + 1, v.y);
            put(row, j + 2, v.z);
            put(row, j + 3, v.w);
        }
    }
    __syncthreads();
    for (int row = warp; row < 16; row += kFewThreads / 32) {
        float m = 0.f;
        for (int j = lane; j < W; j += 32) m = fmaxf(m, row < cnt && j < p.R ? finite_or_0(s_z[row][j]) : 0.f);
        float inv;
        const float c = norm_scale(warp_max(m), inv);
        for (int j = lane; j < W; j += 32) {
            store_pieces(row < cnt && j < p.R ? s_z[row][j] * c : 0.f, &s_p[0][row][j], 16 * W);
        }
        if (lane == 0) s_scale[row] = inv;
    }
    __syncthreads();
    float acc[4][4] = {};
#pragma unroll
    for (int k = 0; k < KB; ++k) {
        const int j = k * 16 + tig * 4;
#pragma unroll
        for (int l = 0; l < kPieces<TX>; ++l) {
            const uint2 z0 = *reinterpret_cast<const uint2 *>(&s_p[l][g][j]);
            const uint2 z1 = *reinterpret_cast<const uint2 *>(&s_p[l][g + 8][j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_t<TX>(acc[i], z0.x, z1.x, z0.y, z1.y, bv[i][k].x, bv[i][k].y);
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (rows[r] < 0) continue;
        const float sc = s_scale[g + 8 * r];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = n0 + i * 8 + tig * 2 + e;
                if (n < p.N)
                    y[rows[r] * p.ldy + n] = from_f32<TY>(fmaf(acc[i][2 * r + e] * sc, scaling, yv[r][i][e]));
            }
    }
}

// ============================================================================ tiles
// Ring of shared-memory stages between the load warps and the thread that issues the MMAs.
// A load thread copies its share of a stage's rows with cp.async (a tile's tokens lie
// anywhere; row gathers by TMA were slower: 26 against 21 us for the shrink of 4096 tokens of
// 6144) and leaves an arrival behind that follows the copies; the weights' boxes come by TMA
// and add one arrival.  The MMA thread makes the copies visible to the tensor core.
//
// The tensor core adds to its fp32 accumulators with truncation, an error that grows with
// the number of additions (weight gradients over 1000 bf16 tokens were off by 2e-6, plain
// fp32 sums by 9e-7), so a chain of kChain steps (16 MMAs) ends in a drain: the load warps
// add the accumulators to registers, rounding to nearest, while the next chain runs in the
// other set of columns (`sets` of them; with one the next chain waits).  4.2e-7 with 16 MMAs
// a chain, 7.8e-7 with 32, in the same time.
constexpr int kChain = 4;

template <int NS>
struct Ring {
    uint64_t full[NS], empty[NS], chain[2], drained[2];
    __device__ void init()
    {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], kWorkers + 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&chain[i], 1);
            mbar_init(&drained[i], kWorkers / 32);
        }
        fence_mbar_init();
    }
};

// Load loop of one thread: copy(stage, i) starts the copies of step i, add(set) adds the
// accumulators of a complete chain.
template <int NS, typename F, typename G>
__device__ __forceinline__ void ring_load(Ring<NS> &r, int steps, int sets, int *status, F &&copy, G &&add)
{
    bool ok = true;
    auto drain = [&](int g) {
        const int set = g & (sets - 1);
        ok = ok && mbar_wait(&r.chain[set], (g >> (sets - 1)) & 1, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_after();
        add(set);
        tc_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&r.drained[set]);
    };
    int g = 0;
    for (int i = 0; i < steps && ok; ++i) {
        if (i >= NS) ok = mbar_wait(&r.empty[i % NS], ((i / NS) & 1) ^ 1, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        copy(i % NS, i);
        cp_async_arrive(&r.full[i % NS]);
        if (i == (g + 1) * kChain + NS - 1) drain(g++);   // (its MMAs are complete: the stage is free)
    }
    for (; g * kChain < steps && ok; ++g) drain(g);
    cp_async_wait<0>();
}

// Issue loop of the MMA thread: mma(stage, set, fresh) issues the MMAs of a step, the first of
// them overwriting the accumulators if fresh.
template <int NS, typename F>
__device__ __forceinline__ void ring_mma(Ring<NS> &r, int steps, int sets, int *status, F &&mma)
{
    for (int i = 0; i < steps; ++i) {
        const int g = i / kChain, set = g & (sets - 1);
        const bool fresh = i % kChain == 0;
        if (fresh && g >= sets && !mbar_wait(&r.drained[set], ((g >> (sets - 1)) & 1) ^ 1, status)) return;
        if (!mbar_wait(&r.full[i % NS], (i / NS) & 1, status)) return;
        fence_async_smem();
        tc_after();
        mma(i % NS, set, fresh);
        tc_commit(&r.empty[i % NS]);
        if (i % kChain == kChain - 1 || i == steps - 1) tc_commit(&r.chain[set]);
    }
}

__device__ __forceinline__ uint32_t tmem_cols(int n) { return n <= 32 ? 32u : n <= 64 ? 64u : n <= 128 ? 128u : n <= 256 ? 256u : 512u; }

constexpr int kShrinkNS = 4;

__host__ __device__ inline int shrink_w_bytes(bool grad, int R, int Kp)
{
    return grad ? (R > 64 ? 2 : 1) * 64 * 128 : Kp * 128;   // multiples of 1024
}

// z = X A^T of one tile of 128 tokens (kGrad: dz = s dY B), K split over the CTAs of a
// cluster.  Operands: X [128 tokens][64 K] K-major; A [ranks][64 K] K-major, or B [64 n][ranks]
// MN-major.  The partial sums meet in shared memory: each CTA adds 128 / S rows of all S
// parts in rank order and writes them: z (fp32), z as pieces with the row's scale, and for
// the weight gradients the adapters' largest magnitudes (fp16) or z_in's pieces (bf16).
// Bound by the rows of X.
template <typename TX, bool kGrad, int KC>   // ranks padded to 16 fit KC columns
__global__ void __launch_bounds__(kTcThreads, KC <= 64 ? 2 : 1)
    shrink_tile_kernel(const __grid_constant__ CUtensorMap map_w, const AdParams p)
{
    extern __shared__ unsigned char raw[];
    __shared__ Ring<kShrinkNS> ring;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) int s_tok[kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = cluster_size(), q = cluster_rank(), tile = blockIdx.x / S;
    unsigned char *buf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    pdl_wait();
    pdl_trigger();
    const int32_t *entry = p.entry_of + (size_t)tile * kTile;
    const int bin = __ldcg(p.tile_bin + tile);
    if (tid < kTile) s_tok[tid] = __ldcg(entry + tid);   // (the tile is inside the plan's arrays)
    if (bin < 0) return;   // (the whole cluster)
    const int rank = rank_of(p, bin), R = p.R, Kp = p.Kp;
    if (rank == 0) {
        if (p.z_out)
            for (int i = q * kTcThreads + tid; i < kTile * R; i += S * kTcThreads) {
                const int t = __ldcg(entry + i / R);
                if (t >= 0) p.z_out[(size_t)t * R + i % R] = 0.f;
            }
        return;
    }
    if (tid == 0) ring.init();
    if (warp == kMmaWarp) tc_alloc(&s_tmem, tmem_cols(2 * Kp));
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem, sbuf = smem_u32(buf);
    const int width = kGrad ? p.N : p.K;
    const int blocks = (width + 63) / 64;
    const int b_lo = (int)((long long)blocks * q / S), steps = (int)((long long)blocks * (q + 1) / S) - b_lo;
    const int wb = shrink_w_bytes(kGrad, R, Kp), stage = kBlk + wb;
    const int pitch = Kp + 4;   // floats of a row of the partial sums
    if (warp < kMmaWarp) {
        const int c = tid & 7, r0 = tid >> 3;
        const TX *X = static_cast<const TX *>(kGrad ? p.dy : p.x);
        const long long ld = kGrad ? p.lddy : p.ldx;
        const TX *px[4];
        bool live[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = s_tok[r0 + 32 * i];
            live[i] = t >= 0;
            px[i] = X + (live[i] ? t * ld : 0) + c * 8;
        }
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int half = warp >> 2;   // of the columns
        float acc[KC / 2] = {};
        ring_load<kShrinkNS>(ring, steps, 2, p.status, [&](int s, int i) {
            const int k0 = (b_lo + i) * 64;
            const uint32_t xs = sbuf + s * stage, ws = xs + kBlk;
            if (tid == 0) {
                mbar_arrive_expect_tx(&ring.full[s], wb);
                if (kGrad) {
                    tma_box(ws, &map_w, &ring.full[s], 0, k0, bin);
                    if (R > 64) tma_box(ws + 8192, &map_w, &ring.full[s], 64, k0, bin);
                } else {
                    tma_box(ws, &map_w, &ring.full[s], k0, 0, bin);
                }
            }
            const bool in = k0 + c * 8 < width;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                cp_async16_or_zero(xs + swz(r0 + 32 * u, c), live[u] && in ? px[u] + k0 : X, live[u] && in);
        }, [&](int set) {
#pragma unroll
            for (int b = 0; b < KC / 2; b += 8) {
                if (b >= Kp / 2) break;
                float v[8];
                tc_ld(tmem + lanes + set * Kp + half * (Kp / 2) + b, v);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[b + e] += v[e];
            }
        });
        float *P = reinterpret_cast<float *>(buf) + ((warp & 3) * 32 + lane) * pitch + half * (Kp / 2);
#pragma unroll
        for (int b = 0; b < KC / 2; b += 4) {
            if (b >= Kp / 2) break;
            *reinterpret_cast<float4 *>(P + b) = make_float4(acc[b], acc[b + 1], acc[b + 2], acc[b + 3]);
        }
    } else if (lane == 0) {
        const uint32_t idesc = idesc16<TX>(Kp, false, kGrad);
        ring_mma<kShrinkNS>(ring, steps, 2, p.status, [&](int s, int set, bool fresh) {
            const uint32_t xs = sbuf + s * stage, ws = xs + kBlk;
            const uint64_t da = sdesc_k(xs), db = kGrad ? sdesc_mn(ws, 8192) : sdesc_k(ws);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                tc_mma16(tmem + set * Kp, da + 2 * kk, db + (kGrad ? 128 : 2) * kk, idesc, !fresh || kk > 0);
        });
    }
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
    if (warp == kMmaWarp) {
        tc_after();
        tc_dealloc(tmem, tmem_cols(2 * Kp));
    } else if (warp < kMmaWarp) {
        const float scaling = kGrad ? __ldcg(p.scaling + bin) : 1.f;
        const float apply_scale = kGrad ? 1.f : __ldcg(p.scaling + bin);
        constexpr int NI = KC / 32;   // columns of a lane
        // one row: lanes over columns
        auto sum = [&](int r, float (&v)[NI]) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int col = lane + 32 * i;
                const uint32_t at = sbuf + (uint32_t)(r * pitch + col) * 4;
                float part[kMaxSplit];
#pragma unroll
                for (int c = 0; c < kMaxSplit; ++c) part[c] = col < Kp && c < S ? ld_cluster(peer_addr(at, c)) : 0.f;
                v[i] = 0.f;
#pragma unroll
                for (int c = 0; c < kMaxSplit; ++c) v[i] += part[c];
            }
        };
        auto finish = [&](int r, float (&v)[NI]) {
            const int tok = s_tok[r];
            const size_t pos = (size_t)tile * kTile + r;
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                v[i] = lane + 32 * i < rank && tok >= 0 ? v[i] * scaling : 0.f;   // (what lies past the rank is not used)
                m = fmaxf(m, finite_or_0(v[i]));
            }
            m = warp_max(m);
            float inv;
            const float c = norm_scale(m, inv);
            TX *pieces = static_cast<TX *>(p.pieces) + pos * kPieces<TX> * Kp;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int col = lane + 32 * i;
                if (col >= Kp) continue;
                store_pieces(v[i] * (TcType<TX>::code ? 1.f : c), pieces + col, Kp);   // (bf16 has fp32's range)
                if (p.z_out && tok >= 0 && col < R) p.z_out[(size_t)tok * R + col] = v[i];
                if (kGrad && p.want_dw && !TcType<TX>::code && col < R) p.dz[pos * R + col] = v[i];
            }
            if (lane == 0) p.row_scale[pos] = (TcType<TX>::code ? 1.f : inv) * apply_scale;
            if (kGrad && p.want_dw) {
                float zm = 0.f;
                TX *zl = static_cast<TX *>(p.zl) + pos * kPieces<TX> * Kp;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int col = lane + 32 * i;
                    const float z = col < rank && tok >= 0 ? __ldcg(p.z_in + (size_t)tok * R + col) : 0.f;
                    if (TcType<TX>::code) {
                        if (col < Kp) store_pieces(z, zl + col, Kp);
                    } else {
                        zm = fmaxf(zm, finite_or_0(z));
                    }
                }
                if (!TcType<TX>::code) {
                    zm = warp_max(zm);
                    if (lane == 0) {   // (a maximum of non-negative floats is one of their bits: any order)
                        atomicMax(p.amax + bin, __float_as_uint(m));
                        atomicMax(p.amax + p.n + bin, __float_as_uint(zm));
                    }
                }
            }
        };
        if (S == kMaxSplit) {   // two rows a warp: both read, then the peers are free
            float v[2][NI];
            sum(q * 16 + warp, v[0]);
            sum(q * 16 + 8 + warp, v[1]);
            cluster_done_reading();
            finish(q * 16 + warp, v[0]);
            finish(q * 16 + 8 + warp, v[1]);
        } else {
            const int per = kTile / S;
            for (int r = q * per + warp; r < (q + 1) * per; r += kWorkers / 32) {
                float v[NI];
                sum(r, v);
                finish(r, v);
            }
            if (S > 1) cluster_done_reading();
        }
    }
    if (S > 1) {
        if (warp == kMmaWarp) cluster_done_reading();
        cluster_wait_readers();   // no CTA leaves while a peer reads its sums
    }
}

// fp16 pools: dz and z as pieces under one scale per adapter (a sum over tokens has no
// place for a scale per token), positions in order, a warp each.
__global__ void __launch_bounds__(kWorkers) pieces_kernel(const AdParams p)
{
    const int lane = threadIdx.x & 31;
    const size_t pos = (size_t)blockIdx.x * (kWorkers / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    const int bin = __ldcg(p.tile_bin + pos / kTile);
    if (bin < 0) return;
    const int rank = rank_of(p, bin);
    if (rank == 0) return;
    const int tok = __ldcg(p.entry_of + pos);
    float inv;
    const float cd = norm_scale(__uint_as_float(__ldcg(p.amax + bin)), inv);
    const float cz = norm_scale(__uint_as_float(__ldcg(p.amax + p.n + bin)), inv);
    const size_t row = pos * kPieces<__half> * p.Kp;
    __half *dl = static_cast<__half *>(p.dl) + row, *zl = static_cast<__half *>(p.zl) + row;
    for (int col = lane; col < p.Kp; col += 32) {
        const bool in = col < rank && tok >= 0;
        store_pieces(in ? __ldcg(p.dz + pos * p.R + col) * cd : 0.f, dl + col, p.Kp);
        store_pieces(in ? __ldcg(p.z_in + (size_t)tok * p.R + col) * cz : 0.f, zl + col, p.Kp);
    }
}

// da[a][j][k] = sum_t dz[t][j] x[t][k] and db[a][n][j] = s sum_t z[t][j] dy[t][n]: one product
// D[c][j] = sum_t X[t][c] Z[t][j] over an adapter's tokens, 128 columns c of X per cluster,
// its tokens dealt to the S CTAs 64 at a time.  Both operands are MN-major (rows are
// tokens); Z's pieces lie side by side as the columns of one
// MMA (two MMAs past 256 columns).  The CTAs' parts meet as in the shrink kernel.  Bound by reading X.
__host__ __device__ inline int grad_z_bytes(int cols) { return (cols + 63) / 64 * 8192; }

// accumulator sets: two where two CTAs of an SM can hold them
__host__ __device__ inline int grad_sets(int cols) { return 2 * cols <= 256 ? 2 : 1; }

template <typename TX, int KC, int NS>
__global__ void __launch_bounds__(kTcThreads, KC <= 64 ? 2 : 1)
    grad_tile_kernel(const __grid_constant__ CUtensorMap map_dz, const __grid_constant__ CUtensorMap map_z,
                     const AdParams p)
{
    extern __shared__ unsigned char raw[];
    __shared__ Ring<NS> ring;
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = cluster_size(), q = cluster_rank();
    const int tiles_a = (p.K + 127) / 128, ct = blockIdx.x / S;
    const bool is_b = ct >= tiles_a;
    const int c0 = (is_b ? ct - tiles_a : ct) * 128, width = is_b ? p.N : p.K;
    unsigned char *buf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    pdl_wait();
    pdl_trigger();
    const int R = p.R, Kp = p.Kp, ZC = kPieces<TX> * Kp;
    const int a = p.order ? __ldcg(p.order + blockIdx.y) : blockIdx.y;   // (long units start first)
    const int tokens_a = __ldcg(p.counts + a);
    const size_t pos0 = (size_t)__ldcg(p.seg + a);
    const int rank = rank_of(p, a), cnt = rank ? tokens_a : 0;
    float *out = is_b ? p.db + ((size_t)a * p.N + c0) * R : p.da + (size_t)a * R * p.K + c0;
    const int cols = min(128, width - c0);
    if (cnt == 0) {   // (the whole cluster)
        if (p.accumulate) return;
        if (is_b) {
            for (int i = q * kTcThreads + tid; i < cols * R; i += S * kTcThreads) out[i] = 0.f;
        } else {
            for (int i = q * kTcThreads + tid; i < 128 * R; i += S * kTcThreads)
                if ((i & 127) < cols) out[(size_t)(i >> 7) * p.K + (i & 127)] = 0.f;
        }
        return;
    }
    const int sets = grad_sets(ZC);
    if (tid == 0) ring.init();
    if (warp == kMmaWarp) tc_alloc(&s_tmem, tmem_cols(sets * ZC));
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem, sbuf = smem_u32(buf);
    const int blocks = (cnt + 63) / 64, steps = (blocks - q + S - 1) / S;   // token blocks q, q + S, ..
    const int stage = 2 * 8192 + grad_z_bytes(ZC);
    const int pitch = is_b ? Kp + 4 : 128 + 4;
    float *P = reinterpret_cast<float *>(buf);
    if (warp < kMmaWarp) {
        const TX *X = static_cast<const TX *>(is_b ? p.dy : p.x);
        const CUtensorMap *mz = is_b ? &map_z : &map_dz;
        const long long ld = is_b ? p.lddy : p.ldx;
        const int cx = tid & 15, rx = tid >> 4;   // 16-byte chunk of a row, first of four rows
        const bool in_x = cx * 8 < cols;
        const TX *Xc = X + c0 + cx * 8;
        // the warp's eight tokens of four steps, a lane each, loaded four steps ahead
        auto tokens = [&](int i) {
            const int step = i + (lane >> 3), row = 16 * ((lane >> 1) & 3) + (warp << 1) + (lane & 1);
            return step < steps ? __ldcg(p.entry_of + pos0 + (size_t)(q + step * S) * 64 + row) : -1;
        };
        int ids = tokens(0), next = tokens(4);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int half = warp >> 2;   // of the ranks
        float acc[KC / 2] = {};
        ring_load<NS>(ring, steps, sets, p.status, [&](int s, int i) {
            const uint32_t xs = sbuf + s * stage + (cx >> 3) * 8192, zs = sbuf + s * stage + 2 * 8192;
            if (tid == 0) {
                mbar_arrive_expect_tx(&ring.full[s], stage - 2 * 8192);
                for (int c = 0; c * 64 < ZC; ++c)
                    tma_box2(zs + c * 8192, mz, &ring.full[s], c * 64, (int)pos0 + (q + i * S) * 64);
            }
            if (i && (i & 3) == 0) {
                ids = next;
                next = tokens(i + 4);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = __shfl_sync(0xffffffffu, ids, (i & 3) * 8 + 2 * u + (lane >> 4));
                const bool in = t >= 0 && in_x;
                cp_async16_or_zero(xs + swz(rx + 16 * u, cx & 7), in ? Xc + t * ld : X, in);
            }
        }, [&](int set) {
#pragma unroll
            for (int b = 0; b < KC / 2; b += 8) {
                if (b >= Kp / 2) break;
                float v[kPieces<TX>][8];
#pragma unroll
                for (int l = 0; l < kPieces<TX>; ++l)
                    tc_ld(tmem + lanes + set * ZC + l * Kp + half * (Kp / 2) + b, v[l]);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float sum = v[kPieces<TX> - 1][e];   // (the smallest first)
#pragma unroll
                    for (int l = kPieces<TX> - 2; l >= 0; --l) sum += v[l][e];
                    acc[b + e] += sum;
                }
            }
        });
        const int c = (warp & 3) * 32 + lane;
        if (S == 1 && !is_b) {   // a lane has a column: rows of da are coalesced as they are
            float scale = 1.f;
            if (!TcType<TX>::code) norm_scale(__uint_as_float(__ldcg(p.amax + a)), scale);
#pragma unroll
            for (int b = 0; b < KC / 2; ++b) {
                const int j = half * (Kp / 2) + b;
                if (b >= Kp / 2 || j >= R || c >= cols) break;
                float *dst = out + (size_t)j * p.K + c;
                if (p.accumulate) {
                    if (j < rank) *dst += acc[b] * scale;
                } else {
                    *dst = j < rank ? acc[b] * scale : 0.f;
                }
            }
        } else {
#pragma unroll
            for (int b = 0; b < KC / 2; ++b) {
                if (b >= Kp / 2) break;
                const int j = half * (Kp / 2) + b;
                if (is_b) P[c * pitch + j] = acc[b];
                else P[j * pitch + c] = acc[b];
            }
        }
    } else if (lane == 0 && steps > 0) {
        const uint32_t idesc = idesc16<TX>(min(ZC, 256), true, true), idesc2 = idesc16<TX>(ZC - 256, true, true);
        ring_mma<NS>(ring, steps, sets, p.status, [&](int s, int set, bool fresh) {
            const uint32_t xs = sbuf + s * stage, d = tmem + set * ZC;
            const uint64_t da = sdesc_mn(xs, 8192), db = sdesc_mn(xs + 2 * 8192, 8192);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                tc_mma16(d, da + 128 * kk, db + 128 * kk, idesc, !fresh || kk > 0);
                if (ZC > 256)   // (columns 256 .. start at block 4)
                    tc_mma16(d + 256, da + 128 * kk, db + 4 * 512 + 128 * kk, idesc2, !fresh || kk > 0);
            }
        });
    }
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
    if (warp == kMmaWarp) {
        tc_after();
        tc_dealloc(tmem, tmem_cols(sets * ZC));
    } else if (warp < kMmaWarp && (S > 1 || is_b)) {
        float scale = is_b ? __ldcg(p.scaling + a) : 1.f, inv = 1.f;
        if (!TcType<TX>::code) {
            norm_scale(__uint_as_float(__ldcg(p.amax + (is_b ? p.n : 0) + a)), inv);
            scale *= inv;
        }
        const int per = is_b ? R / 4 : 32;                    // float4 per row of the output
        const int rows = is_b ? cols : R;
        for (int i = q * kWorkers + tid; i < rows * per; i += S * kWorkers) {
            const int row = i / per, c4 = (i % per) * 4;
            if (!is_b && c4 >= cols) continue;                // (K is a multiple of 8)
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t at = sbuf + (uint32_t)(row * pitch + c4) * 4;
            float4 part[kMaxSplit];
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c)
                if (c < S) part[c] = ld_cluster4(peer_addr(at, c));
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c)
                if (c < S) {
                    v.x += part[c].x;
                    v.y += part[c].y;
                    v.z += part[c].z;
                    v.w += part[c].w;
                }
            float *f = &v.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = (is_b ? c4 + e : row) < rank ? f[e] * scale : 0.f;
            float4 *dst = reinterpret_cast<float4 *>(is_b ? out + (size_t)row * R + c4 : out + (size_t)row * p.K + c4);
            if (p.accumulate) {
                float4 o = *dst;
                float *g = &o.x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((is_b ? c4 + e : row) < rank) g[e] += f[e];
                v = o;
            }
            *dst = v;
        }
    }
    __syncwarp();
    if (S > 1) cluster_sync();
}

// y[t][n] = y_in[t][n] + sum_j z[t][j] B[n][j] (kGrad: dx = dx_in + dz A), whose rows are 16-byte
// aligned.  A persistent CTA per SM takes a run of (tile, 256 bytes of columns) items.
// Operands: z's pieces [128 tokens][pieces x Kp] K-major, loaded once per tile; B [columns]
// [ranks] K-major, or A [ranks][columns] MN-major, in a ring; both by TMA; D in TMEM, double
// buffered.  Sixteen epilogue warps (32 tokens x 128 bytes of every second item) turn D's
// rows (a TMEM lane is a token) into whole 128-byte pieces of rows through shared memory and
// add y_in, whose loads run an item ahead, 64 KB per SM, and its lines two items ahead of
// those into L2.  Bound by reading y_in and writing y.  Measured for 4096 tokens of 6144 bf16
// columns, rank 64 (100 MB: 16 us at the copy peak, 21 us for a bare read-add-write kernel of
// that size): 30 us; earlier forms: a lane per token straight to memory 67 us and a lane per
// column 44 us (the load/store unit), TMA row gathers and scatters 62 us (about 75 cycles per
// four rows), eight epilogue warps 34 us (latency).
constexpr int kEpiWarps = 16;
constexpr int kExpandThreads = kEpiWarps * 32 + 96;   // epilogue, MMA, TMA, fix warps
constexpr int kScratch = 4608;                      // bytes of an epilogue warp's block: 32 x 36 or 16 x 68 floats
constexpr int kAnyThreads = kWorkers + 96;
constexpr int kExpandNS = 4;                    // weight stages at most
constexpr int kAnyNS = 3;
constexpr int kMaxRun = 16;                     // tiles that a CTA's run may touch

// pieces that an output's type can tell apart: two carry 16 bits or more of z
template <typename TX, typename TY>
__host__ __device__ constexpr int use_pieces()
{
    return sizeof(TY) == 2 ? 2 : kPieces<TX>;
}

__host__ __device__ inline int expand_z_bytes(int cols) { return (cols + 63) / 64 * kBlk; }
// bytes of a weight stage of n columns of the output
__host__ __device__ inline int expand_w_bytes(bool grad, int Kp, int n) { return grad ? Kp * 2 * n : (Kp + 63) / 64 * n * 128; }

// Zeros the entries [rank, next multiple of 16) of a weight stage of n output columns: rows
// of an MN-major stage, columns of a K-major one.
template <bool kGrad>
__device__ __forceinline__ void zero_past_rank(unsigned char *w, int rank, int Kp, int n, int lane)
{
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int end = (rank + 15) & ~15;
    if (kGrad) {
        const int ch = n / 8;
        for (int e = lane; e < (end - rank) * ch; e += 32) {
            const int j = rank + e / ch, c = e % ch;
            *reinterpret_cast<uint4 *>(w + (c >> 3) * (Kp * 128) + swz(j, c & 7)) = zero;
        }
        return;
    }
    const int c = rank >> 3, rest = rank & 7, c1 = rest ? c + 1 : c;
    for (int row = lane; row < n; row += 32) {
        if (rest) {
            uint4 *q = reinterpret_cast<uint4 *>(w + (c >> 3) * n * 128 + swz(row, c & 7));
            uint4 v = *q;
            uint32_t *f = &v.x;
#pragma unroll
            for (int h = 0; h < 4; ++h) f[h] &= rest >= 2 * h + 2 ? 0xFFFFFFFFu : rest == 2 * h + 1 ? 0xFFFFu : 0u;
            *q = v;
        }
        if (c1 * 8 < end) *reinterpret_cast<uint4 *>(w + (c1 >> 3) * n * 128 + swz(row, c1 & 7)) = zero;
    }
}

// adds to two neighbouring 16-bit elements, or to one fp32
template <typename TY>
__device__ __forceinline__ uint32_t add_pair(uint32_t base, float a, float b);
template <>
__device__ __forceinline__ uint32_t add_pair<__half>(uint32_t base, float a, float b)
{
    const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&base));
    const __half2 r = __floats2half2_rn(f.x + a, f.y + b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <>
__device__ __forceinline__ uint32_t add_pair<__nv_bfloat16>(uint32_t base, float a, float b)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(base << 16) + a,
                                                   __uint_as_float(base & 0xFFFF0000u) + b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <>
__device__ __forceinline__ uint32_t add_pair<float>(uint32_t base, float a, float)
{
    return __float_as_uint(__uint_as_float(base) + a);
}

template <typename TX, typename TY, bool kGrad>
__global__ void __launch_bounds__(kExpandThreads, 1)
    expand_tile_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_z,
                       const AdParams p, const int ns)
{
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t zfull, zempty, wland[kExpandNS], wfull[kExpandNS], wempty[kExpandNS], tfull[2], tempty[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_bin[kMaxRun], s_rank[kMaxRun];
    __shared__ int s_tok[kMaxRun * kTile];
    __shared__ float s_scale[kMaxRun * kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char *buf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    if (tid == 0) {
        mbar_init(&zfull, 1);
        mbar_init(&zempty, 1);
        for (int i = 0; i < ns; ++i) {
            mbar_init(&wland[i], 1);
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], kEpiWarps / 2);
        }
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    if (warp == kEpiWarps) tc_alloc(&s_tmem, 256);
    constexpr int NW = 256 / sizeof(TY), NB = 128 / sizeof(TY);   // columns of an item, of a warp
    constexpr int kUse = use_pieces<TX, TY>();
    const int Kp = p.Kp, width = kGrad ? p.K : p.N;
    const int zb = expand_z_bytes(kUse * Kp), wb = expand_w_bytes(kGrad, Kp, NW);
    const int nt_all = (width + NW - 1) / NW;
    const long long items = (long long)(__ldcg(p.seg + p.n + 1) / kTile) * nt_all;
    const int lo = (int)(items * blockIdx.x / gridDim.x), hi = (int)(items * (blockIdx.x + 1) / gridDim.x);
    // the run's tiles: adapters, ranks, tokens, scales
    const int tile0 = lo / nt_all, run = hi > lo ? (hi - 1) / nt_all - tile0 + 1 : 0;
    for (int i = tid; i < run; i += kExpandThreads) {
        s_bin[i] = __ldcg(p.tile_bin + tile0 + i);
        s_rank[i] = rank_of(p, s_bin[i]);
    }
    for (int i = tid; i < run * kTile; i += kExpandThreads) {
        s_tok[i] = __ldcg(p.entry_of + (size_t)tile0 * kTile + i);
        s_scale[i] = __ldcg(p.row_scale + (size_t)tile0 * kTile + i);
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t zs = smem_u32(buf), ws = zs + zb, tmem = s_tmem;
    const TY *in = static_cast<const TY *>(p.y_in);
    TY *y = static_cast<TY *>(p.y);
    // every role walks the same items; j counts the ones that have a product (stage s of the
    // ring, in its turn `ph`), zc their tiles
    int cur = -1, j = 0, zc = 0, s = 0, ph = 0;
    auto advance = [&] {
        ++j;
        if (++s == ns) s = 0, ph ^= 1;
    };
    if (warp == kEpiWarps + 1) {   // ---- copies of the operands
        if (lane == 0)
            for (int it = lo; it < hi; ++it) {
                const int lt = it / nt_all - tile0, n0 = it % nt_all * NW;
                if (!s_rank[lt]) continue;
                if (j >= ns && !mbar_wait(&wempty[s], ph ^ 1, p.status)) break;
                const uint32_t w = ws + s * wb;
                mbar_arrive_expect_tx(&wland[s], wb);
                if (kGrad) {
                    for (int b = 0; b < NW / 64; ++b) tma_box(w + b * Kp * 128, &map_w, &wland[s], n0 + b * 64, 0, s_bin[lt]);
                } else {
                    tma_box(w, &map_w, &wland[s], 0, n0, s_bin[lt]);
                    if (Kp > 64) tma_box(w + NW * 128, &map_w, &wland[s], 64, n0, s_bin[lt]);
                }
                if (lt != cur) {
                    cur = lt;
                    if (zc && !mbar_wait(&zempty, (zc - 1) & 1, p.status)) break;
                    mbar_arrive_expect_tx(&zfull, zb);
                    for (int b = 0; b * kBlk < zb; ++b)
                        for (int r = 0; r < kTile; r += 64)
                            tma_box2(zs + b * kBlk + r * 128, &map_z, &zfull, b * 64, (tile0 + lt) * kTile + r);
                    ++zc;
                }
                advance();
            }
    } else if (warp == kEpiWarps + 2) {
        // ---- a last K step that the rank does not fill: what lies past the rank becomes zero
        // (the step's z is zero there, but a NaN or an infinity would still spoil the sum)
        // ---- and the y_in of the items two ahead of the epilogue's loads into L2
        int f_it = lo, f_lt = 0, f_nt = lo - tile0 * nt_all;
        auto prefetch = [&] {
            if (!in || f_it >= hi) return;
            const int n = f_nt * NW;
#pragma unroll
            for (int r = 0; r < kTile; r += 32) {
                const int t = s_tok[f_lt * kTile + r + lane];
                if (t < 0) continue;
                const TY *row = in + t * p.ldy_in + n;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
                if (n + NB < width) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + NB));
            }
            ++f_it;
            if (++f_nt == nt_all) f_nt = 0, ++f_lt;
        };
        for (int i = 0; i < 6; ++i) prefetch();
        for (int it = lo; it < hi; ++it) {
            prefetch();
            const int rank = s_rank[it / nt_all - tile0];
            if (!rank) continue;
            const bool ok = mbar_wait(&wland[s], ph, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (rank & 15) {
                zero_past_rank<kGrad>(buf + zb + s * wb, rank, Kp, NW, lane);
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&wfull[s]);
            advance();
        }
    } else if (warp == kEpiWarps) {   // ---- products
        if (lane == 0) {
            const uint32_t idesc = idesc16<TX>(NW, false, kGrad);
            const uint64_t dz0 = sdesc_k(zs), dw0 = kGrad ? sdesc_mn(ws, Kp * 128) : sdesc_k(ws);
            for (int it = lo; it < hi; ++it) {
                const int lt = it / nt_all - tile0, rank = s_rank[lt], b = j & 1;
                if (!rank) continue;
                if (lt != cur) {
                    cur = lt;
                    if (zc) tc_commit(&zempty);   // the tile before is done with z
                    if (!mbar_wait(&zfull, zc & 1, p.status)) break;
                    ++zc;
                }
                if (!mbar_wait(&wfull[s], ph, p.status)) break;
                if (j >= 2 && !mbar_wait(&tempty[b], ((j >> 1) & 1) ^ 1, p.status)) break;
                tc_after();
                const uint64_t dw = dw0 + ((s * wb) >> 4);
                const int steps = (rank + 15) >> 4;
                for (int l = 0; l < kUse; ++l)
                    for (int k = 0; k < steps; ++k) {   // (a 64-column block holds four steps)
                        const int at = l * (Kp >> 4) + k;
                        tc_mma16(tmem + b * 128, dz0 + (at >> 2) * (kBlk >> 4) + (at & 3) * 2,
                                 dw + (kGrad ? 128 * k : (k >> 2) * (NW * 8) + (k & 3) * 2), idesc, at > 0);
                    }
                tc_commit(&wempty[s]);
                tc_commit(&tfull[b]);
                advance();
            }
        }
    } else {
        // ---- epilogue: tokens [32 q4, +32), 128 bytes of columns of every second item with a
        // product (and of the others), so that sixteen warps hide one another's latencies
        const int q4 = warp & 3, half = (warp >> 2) & 1, group = warp >> 3;
        constexpr int CE = 16 / sizeof(TY);               // elements of a lane's access: 8 lanes, 128 bytes a row
        constexpr int NP = NB / 32, RP = 32 / NP;         // passes, their rows
        constexpr int NA = RP / 4;                        // accesses of a pass, four rows each
        constexpr int kPitch = NB + 4;                    // floats of a row of the warp's block
        float *sc = reinterpret_cast<float *>(buf + zb + ns * wb + warp * kScratch);
        const int rl = lane >> 3, cl = half * NB + (lane & 7) * CE;
        struct Item {
            int it, lt, nt, j;
        };
        // the next item of this group at or behind i
        auto own = [&](Item &i) {
            while (i.it < hi) {
                const bool product = s_rank[i.lt] > 0;
                if (((product ? i.j : i.it) & 1) == group) return;
                i.j += product;
                ++i.it;
                if (++i.nt == nt_all) i.nt = 0, ++i.lt;
            }
        };
        auto behind = [&](Item i) {
            i.j += s_rank[i.lt] > 0;
            ++i.it;
            if (++i.nt == nt_all) i.nt = 0, ++i.lt;
            own(i);
            return i;
        };
        uint4 pre[NP][NA];
        auto fetch = [&](const Item &i, int ps, int a) {
            const int n = i.nt * NW + cl;
            if (!in || i.it >= hi || n >= width) return;
            const int t = s_tok[i.lt * kTile + q4 * 32 + ps * RP + a * 4 + rl];
            if (t >= 0) pre[ps][a] = *reinterpret_cast<const uint4 *>(in + t * p.ldy_in + n);
        };
        Item at = {lo, 0, lo - tile0 * nt_all, 0};
        own(at);
#pragma unroll
        for (int ps = 0; ps < NP; ++ps)
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                pre[ps][a] = make_uint4(0u, 0u, 0u, 0u);
                fetch(at, ps, a);
            }
        int turn = 0;
        while (at.it < hi) {
            const Item next = behind(at);
            const bool product = s_rank[at.lt] > 0;
            float scale = 0.f;
            if (product) {
                const bool ok = mbar_wait(&tfull[group], turn, p.status);
                if (!__all_sync(0xffffffffu, ok)) break;
                turn ^= 1;
                tc_after();
                scale = s_scale[at.lt * kTile + q4 * 32 + lane];
            }
#pragma unroll
            for (int ps = 0; ps < NP; ++ps) {
                if (product) {
#pragma unroll
                    for (int h = 0; h < NB; h += 16) {
                        float v[16];
                        tc_ld(tmem + ((uint32_t)(q4 * 32) << 16) + group * 128 + half * NB + h, v);
                        tc_wait_ld();
                        if (lane / RP == ps)   // (a 16-bit row's 128 bytes are 64 columns: 16 rows at a time)
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<float4 *>(sc + (lane & (RP - 1)) * kPitch + h + e) =
                                    make_float4(v[e] * scale, v[e + 1] * scale, v[e + 2] * scale, v[e + 3] * scale);
                    }
                    tc_before();
                    __syncwarp();
                    if (ps == NP - 1 && lane == 0) mbar_arrive(&tempty[group]);
                }
                const int n = at.nt * NW + cl;
#pragma unroll
                for (int a = 0; a < NA; ++a) {
                    uint4 o = pre[ps][a];
                    if (product) {
                        const float *d = sc + (a * 4 + rl) * kPitch + (lane & 7) * CE;
                        uint32_t *f = &o.x;
                        if (sizeof(TY) == 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(d);
                            f[0] = add_pair<TY>(f[0], x.x, 0.f);
                            f[1] = add_pair<TY>(f[1], x.y, 0.f);
                            f[2] = add_pair<TY>(f[2], x.z, 0.f);
                            f[3] = add_pair<TY>(f[3], x.w, 0.f);
                        } else {   // (a row's last four lanes take their halves in turn: no bank twice)
                            const int h = lane & 4;
                            const float4 u = *reinterpret_cast<const float4 *>(d + h);
                            const float4 w = *reinterpret_cast<const float4 *>(d + (h ^ 4));
                            const float4 x = h ? w : u, z = h ? u : w;
                            f[0] = add_pair<TY>(f[0], x.x, x.y);
                            f[1] = add_pair<TY>(f[1], x.z, x.w);
                            f[2] = add_pair<TY>(f[2], z.x, z.y);
                            f[3] = add_pair<TY>(f[3], z.z, z.w);
                        }
                    }
                    const int t = s_tok[at.lt * kTile + q4 * 32 + ps * RP + a * 4 + rl];
                    if (t >= 0 && n < width && (product || in != y)) *reinterpret_cast<uint4 *>(y + t * p.ldy + n) = o;
                    fetch(next, ps, a);
                }
                __syncwarp();
            }
            at = next;
        }
        tc_before();
    }
    __syncthreads();
    if (warp == kEpiWarps) {
        tc_after();
        tc_dealloc(tmem, 256);
    }
}

// The same for rows of any element alignment, a CTA per tile and run of 128-column blocks.
// The product is D[n][t]: a TMEM lane is a column of y, so a warp's 32 lanes touch
// neighbouring elements of a token's row without passing through shared memory.

// The base's bits of a tile's tokens (zeros without a base), eight accesses in flight
template <typename C, typename TY>
__device__ void copy_rows(const int *tok, const TY *in, long long ld_in, TY *y, long long ldy, int cols)
{
    constexpr int CE = sizeof(C) / sizeof(TY), kU = 8;
    const int per = cols / CE, n = kTile * per;
    for (int e0 = threadIdx.x; e0 < n; e0 += kU * kAnyThreads) {
        C v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int e = e0 + u * kAnyThreads, t = e < n ? tok[e / per] : -1;
            v[u] = C{};
            if (in && t >= 0) v[u] = *reinterpret_cast<const C *>(in + t * ld_in + e % per * CE);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int e = e0 + u * kAnyThreads, t = e < n ? tok[e / per] : -1;
            if (t >= 0) *reinterpret_cast<C *>(y + t * ldy + e % per * CE) = v[u];
        }
    }
}

// kPair: rows of 16-bit elements start at 4-byte boundaries, and two lanes share a 4-byte
// access of neighbouring columns (one takes the even token, the other the odd one)
template <typename TX, typename TY, bool kGrad, bool kPair>
__global__ void __launch_bounds__(kAnyThreads, 2)
    expand_any_kernel(const __grid_constant__ CUtensorMap map, const AdParams p)
{
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t landed[kAnyNS], full[kAnyNS], empty[kAnyNS], tfull[2], tempty[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_tok[kTile];
    __shared__ __align__(16) float s_scale[kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tile = blockIdx.x;
    unsigned char *buf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    pdl_wait();
    pdl_trigger();
    const int bin = __ldcg(p.tile_bin + tile);
    if (bin < 0) return;
    const int rank = rank_of(p, bin), Kp = p.Kp, ZC = kPieces<TX> * Kp, width = kGrad ? p.K : p.N;
    const int nt_all = (width + 127) / 128;
    const int nt0 = (int)((long long)nt_all * blockIdx.y / gridDim.y);
    const int nts = (int)((long long)nt_all * (blockIdx.y + 1) / gridDim.y) - nt0;
    const TY *in = static_cast<const TY *>(p.y_in);
    TY *y = static_cast<TY *>(p.y);
    if (tid < kTile) s_tok[tid] = __ldcg(p.entry_of + (size_t)tile * kTile + tid);
    if (rank == 0) {
        if (in == y) return;   // in place: nothing to add
        __syncthreads();
        const int lo = nt0 * 128, cols = min((nt0 + nts) * 128, width) - lo;
        auto wide = [](const void *q, long long ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * sizeof(TY) % 16 == 0; };
        if (wide(y, p.ldy) && (!in || wide(in, p.ldy_in)) && cols * sizeof(TY) % 16 == 0)
            copy_rows<uint4, TY>(s_tok, in ? in + lo : nullptr, p.ldy_in, y + lo, p.ldy, cols);
        else
            copy_rows<typename std::conditional<sizeof(TY) == 4, uint32_t, uint16_t>::type, TY>(
                s_tok, in ? in + lo : nullptr, p.ldy_in, y + lo, p.ldy, cols);
        return;
    }
    const uint32_t zs = smem_u32(buf), ws = zs + expand_z_bytes(ZC), wb = expand_w_bytes(kGrad, Kp, 128);
    const bool fix = rank & 15;
    if (tid == 0) {
        for (int i = 0; i < kAnyNS; ++i) {
            mbar_init(&landed[i], 1);
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], kWorkers / 32);
        }
        fence_mbar_init();
    }
    if (warp == kWorkers / 32) tc_alloc(&s_tmem, 256);
    if (warp < kWorkers / 32) {   // z's pieces: chunk c of a row is columns 8 c ..
        const TX *Z = static_cast<const TX *>(p.pieces) + (size_t)tile * kTile * ZC;
        const int ch = ZC / 8;
        for (int c = tid & 7; c < ch; c += 8)
            for (int row = tid >> 3; row < kTile; row += kWorkers / 8)
                cp_async16_or_zero(zs + (c >> 3) * kBlk + swz(row, c & 7), Z + (size_t)row * ZC + c * 8, true);
        if (tid < kTile) s_scale[tid] = __ldcg(p.row_scale + (size_t)tile * kTile + tid);
        cp_async_commit();
        cp_async_wait<0>();
        fence_async_smem();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    if (warp == kWorkers / 32 + 1) {   // ---- weights
        // ---- and the next block's y_in into L2: what the epilogue's registers can keep in
        // flight covers the latency of L2, not of HBM
        int tok[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) tok[u] = s_tok[lane + 32 * u];
        auto prefetch = [&](int i) {
            const int n0 = (nt0 + i) * 128;
            if (!in || i >= nts) return;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < 128; c += 128 / (int)sizeof(TY))
                    if (tok[u] >= 0 && n0 + c < width)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(in + tok[u] * p.ldy_in + n0 + c));
        };
        prefetch(0);
        prefetch(1);
        for (int i = 0; i < nts; ++i) {
            const int s = i % kAnyNS, n0 = (nt0 + i) * 128;
            const uint32_t w = ws + s * wb;
            bool ok = true;
            if (i >= kAnyNS) ok = mbar_wait(&empty[s], ((i / kAnyNS) & 1) ^ 1, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&landed[s], wb);
                if (kGrad) {
                    tma_box(w, &map, &landed[s], n0, 0, bin);
                    tma_box(w + Kp * 128, &map, &landed[s], n0 + 64, 0, bin);
                } else {
                    tma_box(w, &map, &landed[s], 0, n0, bin);
                    if (Kp > 64) tma_box(w + kBlk, &map, &landed[s], 64, n0, bin);
                }
            }
            prefetch(i + 2);
        }
    } else if (warp == kWorkers / 32 + 2) {
        // ---- a last K step that the rank does not fill: what lies past the rank becomes zero
        // (the step's z is zero there, but a NaN or an infinity would still spoil the sum)
        for (int i = 0; fix && i < nts; ++i) {
            const int s = i % kAnyNS;
            const bool ok = mbar_wait(&landed[s], (i / kAnyNS) & 1, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            zero_past_rank<kGrad>(buf + (ws - zs) + s * wb, rank, Kp, 128, lane);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
    } else if (warp == kWorkers / 32) {   // ---- products
        if (lane == 0) {
            const uint32_t idesc = idesc16<TX>(128, kGrad, false);
            for (int i = 0; i < nts; ++i) {
                const int s = i % kAnyNS, b = i & 1;
                if (!mbar_wait(fix ? &full[s] : &landed[s], (i / kAnyNS) & 1, p.status)) break;
                if (i >= 2 && !mbar_wait(&tempty[b], ((i >> 1) & 1) ^ 1, p.status)) break;
                tc_after();
                const uint32_t w = ws + s * wb;
                for (int l = 0; l < use_pieces<TX, TY>(); ++l)   // (as above: the same bits)
                    for (int j = 0; j < rank; j += 16) {
                        const int at = l * Kp + j;
                        const uint64_t dw = kGrad ? sdesc_mn(w, Kp * 128) + 8 * j : sdesc_k(w + (j >> 6) * kBlk) + ((j & 63) >> 3);
                        const uint64_t dz = sdesc_k(zs + (at >> 6) * kBlk) + ((at & 63) >> 3);
                        tc_mma16(tmem + b * 128, dw, dz, idesc, at > 0);
                    }
                tc_commit(&empty[s]);
                tc_commit(&tfull[b]);
            }
        }
    } else {   // ---- epilogue: tokens [64 half, +64) of columns [32 q4, +32)
        const int q4 = warp & 3, half = warp >> 2;
        constexpr bool kTwo = kPair && sizeof(TY) == 2;   // two tokens per access
        constexpr int GT = 8, NG = 64 / GT;               // tokens of a group, groups of a block
        constexpr int kAcc = kTwo ? 4 : 8;                // accesses of a group
        constexpr int kAhead = kTwo ? 4 : 2;              // groups in flight: 2 KB a warp
        const int odd = kTwo ? lane & 1 : 0;
        const int col = q4 * 32 + (kTwo ? lane & ~1 : lane);
        using V = typename std::conditional<kTwo || sizeof(TY) == 4, uint32_t, uint16_t>::type;
        V pre[kAhead][kAcc];
        auto fetch = [&](int g, V (&v)[kAcc]) {   // group g of the run
            const int n = (nt0 + g / NG) * 128 + col;
#pragma unroll
            for (int a = 0; a < kAcc; ++a) {
                const int t = s_tok[half * 64 + g % NG * GT + (kTwo ? 2 * a + odd : a)];
                v[a] = 0;
                if (in && g < NG * nts && t >= 0 && n < width) v[a] = *reinterpret_cast<const V *>(in + t * p.ldy_in + n);
            }
        };
#pragma unroll
        for (int g = 0; g < kAhead; ++g) fetch(g, pre[g]);
        for (int i = 0; i < nts; ++i) {
            const int b = i & 1, n = (nt0 + i) * 128 + col;
            const bool ok = mbar_wait(&tfull[b], (i >> 1) & 1, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_after();
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int t0 = half * 64 + g * GT;
                float v[GT];
                tc_ld(tmem + ((uint32_t)(q4 * 32) << 16) + b * 128 + t0, v);
                tc_wait_ld();
                if (g == NG - 1) {
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[b]);
                }
#pragma unroll
                for (int e = 0; e < GT; e += 4) {
                    const float4 sc = *reinterpret_cast<const float4 *>(s_scale + t0 + e);
                    v[e] *= sc.x;
                    v[e + 1] *= sc.y;
                    v[e + 2] *= sc.z;
                    v[e + 3] *= sc.w;
                }
                V o[kAcc];
#pragma unroll
                for (int a = 0; a < kAcc; ++a) {
                    if (kTwo) {   // my token's value of my column, and of my neighbour's
                        const float mine = odd ? v[(2 * a + 1) % GT] : v[2 * a % GT];
                        const float theirs = __shfl_xor_sync(0xffffffffu, odd ? v[2 * a % GT] : v[(2 * a + 1) % GT], 1);
                        o[a] = add_pair<TY>(pre[g % kAhead][a], odd ? theirs : mine, odd ? mine : theirs);
                    } else if (sizeof(TY) == 4) {
                        o[a] = add_pair<float>(pre[g % kAhead][a], v[a], 0.f);
                    } else {
                        const TY base = *reinterpret_cast<const TY *>(&pre[g % kAhead][a]);
                        const TY r = from_f32<TY>(f32_of(base) + v[a]);
                        o[a] = *reinterpret_cast<const V *>(&r);
                    }
                }
                fetch(NG * i + g + kAhead, pre[g % kAhead]);
#pragma unroll
                for (int a = 0; a < kAcc; ++a) {
                    const int t = s_tok[t0 + (kTwo ? 2 * a + odd : a)];
                    if (t >= 0 && n < width) *reinterpret_cast<V *>(y + t * p.ldy + n) = o[a];
                }
            }
        }
        tc_before();
    }
    __syncthreads();
    if (warp == kWorkers / 32) {
        tc_after();
        tc_dealloc(tmem, 256);
    }
}

// ============================================================================ host
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype >= MOE_DTYPE_F16 && dtype <= MOE_DTYPE_F32; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int tiles_max(const moe_adapters_desc &d, int T) { return (T + kTile - 1) / kTile + std::min(d.n_adapters + 1, T); }
int few_splits(const moe_adapters_desc &d) { return (d.in_features + kFewK - 1) / kFewK; }
int pieces_of(const moe_adapters_desc &d) { return d.dtype == MOE_DTYPE_BF16 ? kPieces<__nv_bfloat16> : kPieces<__half>; }
int rank_pad(const moe_adapters_desc &d) { return (d.max_rank + 15) / 16 * 16; }

// a call's workspace: the small path's partial sums share the bytes of the other path
struct AdWs {
    size_t seg, counts, entry_of, tile_bin, order, hist, pieces, row_scale, zl, dl, dz, amax, total;
};

AdWs ad_layout(const moe_adapters_desc &d, int T)
{
    AdWs w;
    const size_t bins = d.n_adapters + 1, tiles = tiles_max(d, T), rows = tiles * kTile;
    const size_t pieces = rows * pieces_of(d) * rank_pad(d) * 2;
    size_t o = 0;
    w.seg = o; o = up256(o + (bins + 1) * 4);
    w.counts = o; o = up256(o + bins * 4);
    w.entry_of = o; o = up256(o + rows * 4);
    w.tile_bin = o; o = up256(o + tiles * 4);
    w.order = o; o = up256(o + bins * 4);
    w.hist = o; o = up256(o + ((size_t)T + kSortChunk - 1) / kSortChunk * bins * 4);
    w.pieces = o; o = up256(o + pieces);
    w.row_scale = o; o = up256(o + rows * 4);
    w.zl = o; o = up256(o + pieces);
    w.dl = o; o = up256(o + pieces);
    w.dz = o; o = up256(o + rows * d.max_rank * 4);
    w.amax = o; o = up256(o + 2 * bins * 4);
    const size_t few = (size_t)few_splits(d) * std::min(T, kFewT) * d.max_rank * 4;
    w.total = std::max(o, up256(few));
    return w;
}

bool ld_ok(int64_t ld, int width) { return ld >= width && (uint64_t)ld < (1ull << 40); }

// rows of 16-bit elements that 16-byte loads can read
bool rows16_ok(const void *p, int64_t ld, int width) { return p && aligned16(p) && ld_ok(ld, width) && ld % 8 == 0; }

// rows that are read and written element by element, or wider as they are aligned
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

AdParams ad_params(const moe_adapters *h, const int32_t *adapter_of, int T, void *ws)
{
    const moe_adapters_desc &d = h->desc;
    const AdWs w = ad_layout(d, T);
    auto at = [&](size_t off) { return static_cast<char *>(ws) + off; };
    AdParams p = {};
    p.a = h->w.a;
    p.b = h->w.b;
    p.scaling = h->w.scaling;
    p.rank = h->w.rank;
    p.adapter_of = adapter_of;
    p.T = T;
    p.K = d.in_features;
    p.N = d.out_features;
    p.R = d.max_rank;
    p.Kp = rank_pad(d);
    p.n = d.n_adapters;
    p.status = h->d_status;
    p.seg = reinterpret_cast<int32_t *>(at(w.seg));
    p.counts = reinterpret_cast<int32_t *>(at(w.counts));
    p.entry_of = reinterpret_cast<int32_t *>(at(w.entry_of));
    p.tile_bin = reinterpret_cast<int32_t *>(at(w.tile_bin));
    p.order = d.n_adapters <= kOrdered ? reinterpret_cast<int32_t *>(at(w.order)) : nullptr;
    p.pieces = at(w.pieces);
    p.row_scale = reinterpret_cast<float *>(at(w.row_scale));
    p.zl = at(w.zl);
    p.dl = d.dtype == MOE_DTYPE_F16 ? at(w.dl) : at(w.pieces);   // bf16: dz's pieces serve both products
    p.dz = reinterpret_cast<float *>(at(w.dz));
    p.amax = reinterpret_cast<unsigned *>(at(w.amax));
    p.z_part = reinterpret_cast<float *>(ws);
    p.splits = few_splits(d);
    return p;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// 3-D map of a pool's matrices [n][rows][cols] of 16-bit elements, boxes of 64 columns x box
// rows, 128-byte swizzle
bool make_pool_map(CUtensorMap *m, const void *base, int cols, int rows, int n, int box_rows)
{
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * 2 * (cuuint64_t)rows};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map of rows of pieces, boxes of 64 columns x 64 rows
bool make_rows_map(CUtensorMap *m, const void *base, int cols, size_t rows)
{
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {64, 64}, unit[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t run_sort(const moe_adapters *h, const AdParams &p, void *ws, cudaStream_t s)
{
    SortParams q = {};
    q.key = p.adapter_of;
    q.n = p.T;
    q.E = p.n + 1;
    q.align = kTile;
    q.none_bin = p.n;
    q.counts = p.counts;
    q.seg = p.seg;
    q.entry_of = p.entry_of;
    q.tile_bin = p.tile_bin;
    q.order = p.want_dw ? p.order : nullptr;
    q.max_tiles = tiles_max(h->desc, p.T);
    q.zero = p.amax;
    q.n_zero = 2 * p.n;
    q.hist = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + ad_layout(h->desc, p.T).hist);
    q.status = p.status;
    return launch_sort(q, s);
}

// CTAs of a cluster that share `blocks` steps of work so that `units` clusters make `want`
// CTAs: two per SM, not more, as every CTA costs some 4 us beside its steps (weight gradients
// of 4096 tokens, four adapters, 384 units: one CTA a unit 31 us, two 37, four 53)
int split_of(long long units, int blocks, int want)
{
    int S = 1;
    while (S < kMaxSplit && units * S < want && 2 * S <= blocks) S *= 2;
    return S;
}

// rows of pieces, by position
bool make_pieces_map(const moe_adapters *h, CUtensorMap *m, const void *base, int T)
{
    return make_rows_map(m, base, pieces_of(h->desc) * rank_pad(h->desc), (size_t)tiles_max(h->desc, T) * kTile);
}

template <typename TX, bool kGrad>
cudaError_t run_shrink(const moe_adapters *h, const AdParams &p, cudaStream_t s)
{
    const int tiles = tiles_max(h->desc, p.T);
    const int S = split_of(tiles, ((kGrad ? p.N : p.K) + 63) / 64, 2 * h->num_sms);
    const size_t ring = (size_t)kShrinkNS * (kBlk + shrink_w_bytes(kGrad, p.R, p.Kp));
    const size_t sums = (size_t)kTile * (p.Kp + 4) * 4;
    const ChainLaunch l = {dim3(tiles * S), kTcThreads, 1024 + std::max(ring, sums), S, s};
    const auto kernel = p.Kp <= 32   ? shrink_tile_kernel<TX, kGrad, 32>
                        : p.Kp <= 64 ? shrink_tile_kernel<TX, kGrad, 64>
                                     : shrink_tile_kernel<TX, kGrad, 128>;
    return launch_chained(kernel, l, kGrad ? h->map_b64 : h->map_a, p);
}

template <typename TX>
cudaError_t run_grad(const moe_adapters *h, const AdParams &p, cudaStream_t s)
{
    CUtensorMap dz = {}, z = {};
    if (p.T && !(make_pieces_map(h, &dz, p.dl, p.T) && make_pieces_map(h, &z, p.zl, p.T))) return cudaErrorInvalidValue;
    const int tiles = (p.K + 127) / 128 + (p.N + 127) / 128, live = std::max(1, std::min(p.n, p.T));
    const int S = split_of((long long)tiles * live, (p.T / live + 63) / 64, 2 * h->num_sms);
    // stages of 64 tokens: as many as let two CTAs share an SM, or three (ranks above 64)
    const size_t stage = 2 * 8192 + grad_z_bytes(kPieces<TX> * p.Kp);
    const size_t sums = (size_t)std::max(128 * (p.Kp + 4), p.Kp * 132) * 4;
    const int ns = p.Kp > 64 || 3 * stage <= 108 * 1024 ? 3 : 2;
    const ChainLaunch l = {dim3(tiles * S, p.n), kTcThreads, 1024 + std::max(ns * stage, sums), S, s};
    const auto kernel = p.Kp <= 32   ? grad_tile_kernel<TX, 32, 3>
                        : p.Kp > 64  ? grad_tile_kernel<TX, 128, 3>
                        : ns == 3    ? grad_tile_kernel<TX, 64, 3>
                                     : grad_tile_kernel<TX, 64, 2>;
    return launch_chained(kernel, l, dz, z, p);
}

template <typename TX, typename TY, bool kGrad>
cudaError_t run_expand_tiles(const moe_adapters *h, const AdParams &p, cudaStream_t s)
{
    const int tiles = tiles_max(h->desc, p.T), width = kGrad ? p.K : p.N;
    const size_t es = sizeof(TY), zb = expand_z_bytes(kPieces<TX> * p.Kp);
    auto rows16 = [&](const void *q, long long ld) { return !q || (aligned16(q) && ld * es % 16 == 0); };
    CUtensorMap z;
    if (width * es % 16 == 0 && rows16(p.y, p.ldy) && rows16(p.y_in, p.ldy_in) && tiles / h->num_sms + 2 <= kMaxRun) {
        if (!make_pieces_map(h, &z, p.pieces, p.T)) return cudaErrorInvalidValue;
        const size_t wb = expand_w_bytes(kGrad, p.Kp, 256 / es), scratch = kEpiWarps * kScratch;
        const size_t fixed = 1024 + expand_z_bytes(use_pieces<TX, TY>() * p.Kp) + scratch;
        const int ns = (int)std::min<size_t>(kExpandNS, (kMaxSmem - 16 * 1024 - fixed) / wb);   // (16 KB: the run's tiles)
        return launch_chained(expand_tile_kernel<TX, TY, kGrad>, {dim3(h->num_sms), kExpandThreads, fixed + ns * wb, 1, s},
                              kGrad ? h->map_a : es == 4 ? h->map_b64 : h->map_b, z, p, ns);
    }
    const int groups = std::max(1, std::min((width + 127) / 128, 2 * h->num_sms / tiles));
    const size_t smem = 1024 + zb + kAnyNS * (size_t)expand_w_bytes(kGrad, p.Kp, 128);
    auto pairs = [&](const void *q, long long ld) { return reinterpret_cast<uintptr_t>(q) % 4 == 0 && ld % 2 == 0; };
    const bool pair = width % 2 == 0 && pairs(p.y, p.ldy) && (!p.y_in || pairs(p.y_in, p.ldy_in));
    const bool two = sizeof(TY) == 2 && pair;   // (fp32 has no pairs)
    const ChainLaunch l = {dim3(tiles, groups), kAnyThreads, smem, 1, s};
    const CUtensorMap &w = kGrad ? h->map_a : h->map_b;
    return two ? launch_chained(expand_any_kernel<TX, TY, kGrad, sizeof(TY) == 2>, l, w, p)
               : launch_chained(expand_any_kernel<TX, TY, kGrad, false>, l, w, p);
}

template <typename TX, bool kGrad>
cudaError_t run_expand(const moe_adapters *h, const AdParams &p, int y_dtype, cudaStream_t s)
{
    switch (y_dtype) {
    case MOE_DTYPE_F16: return run_expand_tiles<TX, __half, kGrad>(h, p, s);
    case MOE_DTYPE_BF16: return run_expand_tiles<TX, __nv_bfloat16, kGrad>(h, p, s);
    default: return run_expand_tiles<TX, float, kGrad>(h, p, s);
    }
}

template <typename TX, typename TY>
cudaError_t run_few_expand(const AdParams &p, cudaStream_t s)
{
    const ChainLaunch l = {dim3((p.N + kFewN - 1) / kFewN, p.T), kFewThreads, 0, 1, s};
    const int kb = p.Kp / 16;
    if (kb <= 1) return launch_chained(expand_few_kernel<TX, TY, 1>, l, p);
    if (kb <= 2) return launch_chained(expand_few_kernel<TX, TY, 2>, l, p);
    if (kb <= 4) return launch_chained(expand_few_kernel<TX, TY, 4>, l, p);
    return launch_chained(expand_few_kernel<TX, TY, 8>, l, p);
}

template <typename TX>
cudaError_t run_few(const AdParams &p, int y_dtype, cudaStream_t s)
{
    const ChainLaunch l = {dim3(p.splits, p.T), kFewThreads, 0, 1, s};
    const int nb = p.R / 8;
    const cudaError_t e = nb <= 1   ? launch_chained(shrink_few_kernel<TX, 1>, l, p)
                          : nb <= 2 ? launch_chained(shrink_few_kernel<TX, 2>, l, p)
                          : nb <= 4 ? launch_chained(shrink_few_kernel<TX, 4>, l, p)
                          : nb <= 8 ? launch_chained(shrink_few_kernel<TX, 8>, l, p)
                                    : launch_chained(shrink_few_kernel<TX, 16>, l, p);
    if (e != cudaSuccess) return e;
    switch (y_dtype) {
    case MOE_DTYPE_F16: return run_few_expand<TX, __half>(p, s);
    case MOE_DTYPE_BF16: return run_few_expand<TX, __nv_bfloat16>(p, s);
    default: return run_few_expand<TX, float>(p, s);
    }
}

template <typename TX, typename TY>
cudaError_t prepare_expand()
{
    cudaError_t e = allow_smem(expand_tile_kernel<TX, TY, false>);
    if (e == cudaSuccess) e = allow_smem(expand_tile_kernel<TX, TY, true>);
    if (e == cudaSuccess) e = allow_smem(expand_any_kernel<TX, TY, false, false>);
    if (e == cudaSuccess) e = allow_smem(expand_any_kernel<TX, TY, true, false>);
    if (e == cudaSuccess && sizeof(TY) == 2) e = allow_smem(expand_any_kernel<TX, TY, false, sizeof(TY) == 2>);
    if (e == cudaSuccess && sizeof(TY) == 2) e = allow_smem(expand_any_kernel<TX, TY, true, sizeof(TY) == 2>);
    return e;
}

// shared-memory limits of the kernels that a pool's calls launch
template <typename TX>
cudaError_t prepare()
{
    cudaError_t e = cudaSuccess;
    auto allow = [&](auto kernel) {
        if (e == cudaSuccess) e = allow_smem(kernel);
    };
    allow(shrink_tile_kernel<TX, false, 32>);
    allow(shrink_tile_kernel<TX, false, 64>);
    allow(shrink_tile_kernel<TX, false, 128>);
    allow(shrink_tile_kernel<TX, true, 32>);
    allow(shrink_tile_kernel<TX, true, 64>);
    allow(shrink_tile_kernel<TX, true, 128>);
    allow(grad_tile_kernel<TX, 32, 3>);
    allow(grad_tile_kernel<TX, 64, 2>);
    allow(grad_tile_kernel<TX, 64, 3>);
    allow(grad_tile_kernel<TX, 128, 3>);
    if (e == cudaSuccess) e = prepare_expand<TX, __half>();
    if (e == cudaSuccess) e = prepare_expand<TX, __nv_bfloat16>();
    return e == cudaSuccess ? prepare_expand<TX, float>() : e;
}

template <typename TX>
cudaError_t run_apply(const moe_adapters *h, const AdParams &p, int y_dtype, void *ws, cudaStream_t s)
{
    if (p.T <= kFewT) return run_few<TX>(p, y_dtype, s);
    cudaError_t e = run_sort(h, p, ws, s);
    if (e == cudaSuccess) e = run_shrink<TX, false>(h, p, s);
    return e != cudaSuccess ? e : run_expand<TX, false>(h, p, y_dtype, s);
}

template <typename TX>
cudaError_t run_backward(const moe_adapters *h, const AdParams &p, int dx_dtype, void *ws, cudaStream_t s)
{
    cudaError_t e = run_sort(h, p, ws, s);
    if (e == cudaSuccess && p.T) e = run_shrink<TX, true>(h, p, s);
    if (e == cudaSuccess && p.want_dw && p.T && !TcType<TX>::code)
        e = launch_chained(pieces_kernel, {dim3(tiles_max(h->desc, p.T) * (kTile / (kWorkers / 32))), kWorkers, 0, 1, s}, p);
    if (e == cudaSuccess && p.want_dw) e = run_grad<TX>(h, p, s);
    return e != cudaSuccess || !p.y || !p.T ? e : run_expand<TX, true>(h, p, dx_dtype, s);
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
        !make_pool_map(&h->map_a, w.a, d.in_features, d.max_rank, d.n_adapters, rank_pad(d)) ||
        !make_pool_map(&h->map_b, w.b, d.max_rank, d.out_features, d.n_adapters, 128) ||
        !make_pool_map(&h->map_b64, w.b, d.max_rank, d.out_features, d.n_adapters, 64) ||
        (d.dtype == MOE_DTYPE_F16 ? prepare<__half>() : prepare<__nv_bfloat16>()) != cudaSuccess ||
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
    AdParams p = ad_params(h, adapter_of, T, ws);
    p.x = x;
    p.ldx = ldx;
    p.y_in = y_in;
    p.ldy_in = ldy_in;
    p.y = y;
    p.ldy = ldy;
    p.z_out = z;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(d.dtype == MOE_DTYPE_F16 ? run_apply<__half>(h, p, y_dtype, ws, s)
                                                : run_apply<__nv_bfloat16>(h, p, y_dtype, ws, s));
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
    AdParams p = ad_params(h, adapter_of, T, ws);
    p.x = x;
    p.ldx = ldx;
    p.z_in = z;
    p.dy = dy;
    p.lddy = lddy;
    p.y_in = dx_in;
    p.ldy_in = lddx_in;
    p.y = dx;
    p.ldy = lddx;
    p.accumulate = accumulate != 0;
    p.want_dw = da != nullptr;
    p.da = da;
    p.db = db;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(d.dtype == MOE_DTYPE_F16 ? run_backward<__half>(h, p, dx_dtype, ws, s)
                                                : run_backward<__nv_bfloat16>(h, p, dx_dtype, ws, s));
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

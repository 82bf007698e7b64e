// k_ce.cuh -- softmax cross entropy over the outputs of a W4A8 head: what
// surrounds the contractions (k_gemm.cuh holds the epilogues that reduce a
// tile of outputs, or turn it into its gradient, without storing it).
//
//   lse[m] = log sum_n e^y[m, n],   loss[m] = lse[m] - y[m, target[m]]
//
// A row's statistics come as pairs (reference in log2, sum of 2^(y log2 e -
// reference)), one per column slice, [M, slices].
#pragma once

#include "cr_device.cuh"
#include "k_gemm.cuh"

namespace cr {
namespace ce {

constexpr int kThreads = 256;

using gm::join;

// lse and loss from a row's joined statistics and its target's output (the
// latter not used for an ignored or invalid target).  In fp64: a few operations
// per row, and the loss is often a small difference of larger numbers.
__device__ __forceinline__ void finish_row(const float2 a, float tlogit, int64_t t, int64_t ignore, int64_t V,
                                           float *loss, float *lse)
{
    // the references are in units of the fp32 constant that made them
    const double l = (double)a.x / (double)gm::kLog2e + log((double)a.y);
    *lse = (float)l;
    float out = 0.0f;
    if (t != ignore)
        out = (t >= 0 && t < V) ? (float)(l - (double)tlogit) : __int_as_float(0x7FC00000);
    *loss = out;
}

// The whole loss of stored fp32 outputs y [M, V] (a decode batch, whose outputs
// the GEMV wrote): a cluster of eight CTAs per row, an eighth of the row each;
// the first one joins the eight from the others' shared memory, in order.
constexpr int kRowCtas = 8;

__global__ void __cluster_dims__(kRowCtas, 1, 1) __launch_bounds__(kThreads)
    row_loss_kernel(const float *__restrict__ y, int64_t V, const int64_t *__restrict__ targets, int64_t ignore,
                    float *__restrict__ loss, float *__restrict__ lse)
{
    const float kNegInf = __int_as_float(0xFF800000);
    constexpr int kPer = 8;  // columns per thread and step
    __shared__ float2 warp_stat[kThreads / 32];
    __shared__ __align__(8) float2 stat;      // the CTA's statistics
    __shared__ __align__(8) float2 target;    // .x: the target's output, in the CTA that has it
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t m = blockIdx.y, t = targets[m];
    const int rank = (int)cluster_ctarank();
    const int64_t slice = (V + kRowCtas - 1) / kRowCtas, n0 = rank * slice, n1 = n0 + slice < V ? n0 + slice : V;
    const float *row = y + m * V;
    float2 a = make_float2(kNegInf, 0.0f);
    for (int64_t n = n0 + threadIdx.x; n < n1; n += kPer * kThreads) {
        float v[kPer], mx = kNegInf;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t c = n + i * kThreads;
            v[i] = c < n1 ? row[c] : kNegInf;
            if (c == t && c < n1)
                target.x = v[i];
            mx = fmaxf(mx, v[i]);
        }
        float2 b = make_float2(__fmul_rn(mx, gm::kLog2e), 0.0f);
        const float base = b.x == kNegInf ? 0.0f : b.x;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            b.y += gm::ex2(__fmaf_rn(v[i], gm::kLog2e, -base));
        join(a, b);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        join(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, o), __shfl_xor_sync(0xFFFFFFFFu, a.y, o)));
    if ((threadIdx.x & 31) == 0)
        warp_stat[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w)
            join(a, warp_stat[w]);
        stat = a;
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
#pragma unroll
        for (int r = 1; r < kRowCtas; ++r)
            join(a, ld_cluster_f2(mapa_shared(smem_u32(&stat), (uint32_t)r)));
        float tl = 0.0f;
        if (t >= 0 && t < V)
            tl = ld_cluster_f2(mapa_shared(smem_u32(&target), (uint32_t)(t / slice))).x;
        finish_row(a, tl, t, ignore, V, loss + m, lse + m);
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its shared memory may be read
}

// lse and loss from the statistics of a row's slices, a warp per row: the lanes
// take every 32nd slice each and are joined in a fixed order.
__global__ void __launch_bounds__(kThreads) loss_kernel(const float2 *__restrict__ part, int64_t slices, int64_t M,
                                                        const int64_t *__restrict__ targets, int64_t ignore, int64_t V,
                                                        const float *__restrict__ tlogit, float *__restrict__ loss,
                                                        float *__restrict__ lse)
{
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t m = (kThreads / 32) * (int64_t)blockIdx.x + (threadIdx.x >> 5);
    if (m >= M)
        return;
    float2 a = make_float2(__int_as_float(0xFF800000), 0.0f);
#pragma unroll 4
    for (int64_t s = lane; s < slices; s += 32)
        join(a, part[m * slices + s]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        join(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, o), __shfl_xor_sync(0xFFFFFFFFu, a.y, o)));
    if (lane == 0)
        finish_row(a, tlogit[m], targets[m], ignore, V, loss + m, lse + m);
}

// The rows that take part in the loss, gathered: every row's index, quantised
// activations, scale, target, lse and dloss in order, their number in *count,
// and zeros in dx for the others.  A gradient is zero where the target is
// ignored, and a batch of prompts and padding is ignored for a good part: the
// contractions then run over `count` rows.  A CTA takes eight rows, a warp
// each, and counts the valid ones before them itself (at most 64 KB of targets,
// from L2): with 32 rows a CTA, 4096 x 4096 took 24 us cold instead of 12.
constexpr int kCompactRows = kThreads / 32;

struct CompactArgs {
    const int64_t *targets;
    int64_t ignore;
    const int8_t *xq;
    const float *xs, *lse, *dloss;
    int64_t M, K;
    int8_t *c_xq;
    float *c_xs, *c_lse, *c_dloss;
    int64_t *c_targets;
    int *rows, *count;
    uint16_t *dx;
};

__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a)
{
    __shared__ int warp_count[kThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t m0 = kCompactRows * (int64_t)blockIdx.x;
    int n = 0;
#pragma unroll 4
    for (int64_t m = threadIdx.x; m < m0; m += kThreads)
        n += a.targets[m] != a.ignore ? 1 : 0;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0)
        warp_count[w] = n;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i)
        base += warp_count[i];
    const int64_t t = lane < kCompactRows && m0 + lane < a.M ? a.targets[m0 + lane] : a.ignore;
    const uint32_t valid = __ballot_sync(0xFFFFFFFFu, t != a.ignore);
    if (w == 0) {
        if ((valid >> lane) & 1u) {
            const int at = base + __popc(valid & ((1u << lane) - 1u));
            const int64_t m = m0 + lane;
            a.rows[at] = (int)m;
            a.c_targets[at] = t;
            a.c_xs[at] = a.xs[m];
            a.c_lse[at] = a.lse[m];
            a.c_dloss[at] = a.dloss[m];
        }
        if (lane == 0 && m0 + kCompactRows >= a.M)
            *a.count = base + __popc(valid);
    }
    const int64_t m = m0 + w;  // the warp's row
    if (m >= a.M)
        return;
    if ((valid >> w) & 1u) {
        const int64_t at = base + __popc(valid & ((1u << w) - 1u));
        const uint4 *src = reinterpret_cast<const uint4 *>(a.xq + m * a.K);
        uint4 *dst = reinterpret_cast<uint4 *>(a.c_xq + at * a.K);
#pragma unroll 8
        for (int64_t i = lane; i < a.K / 16; i += 32)
            dst[i] = src[i];
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(a.dx + m * a.K);
        for (int64_t i = lane; i < a.K / 8; i += 32)
            dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// The last step of a split contraction: bf16 outputs from the fp32 copies of
// the split tiles, added in order, and (acc given) from the fp32 sums of the
// whole ones; without acc the whole tiles' outputs are in dst already, and only
// the split tiles are visited.  Output row `rows[m]` (m without rows).
struct SumArgs {
    const float *acc;     // [M, K], or null
    const float *copies;  // [copies][bm][256]
    int M, K, bm, kblocks, slots, max_splits, split_tail;
    const int *count, *rows;
    uint16_t *dst;
};

__global__ void __launch_bounds__(kThreads) split_sum_kernel(const SumArgs a)
{
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int M = a.count != nullptr ? min(a.M, __ldcg(a.count)) : a.M;
    const gm::Tiling t(M, a.K, a.kblocks, a.bm, a.slots, a.max_splits, a.split_tail);
    constexpr int kTileQuads = gm::kSlotCols / 4;  // float4s of a copy's row
    const int per_row = a.K / 4;
    const int tile_rows = min(a.bm, M);  // fewer than bm only where all tiles have as many
    const int64_t n4 = a.acc != nullptr ? (int64_t)M * per_row
                                        : (int64_t)(t.units - t.full) / t.splits * tile_rows * kTileQuads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n4; i += (int64_t)gridDim.x * kThreads) {
        int m, k, tile;
        if (a.acc != nullptr) {
            m = (int)(i / per_row);
            k = 4 * (int)(i - (int64_t)m * per_row);
            tile = gm::tile_number(m / a.bm, k / gm::kSlotCols, t.tiles_m, t.tiles_n);
        } else {
            int tm, tn;
            const int r = (int)(i / kTileQuads);  // row among the split tiles' rows
            tile = t.full + r / tile_rows;
            gm::tile_place(tile, t.tiles_m, t.tiles_n, tm, tn);
            m = tm * a.bm + r % tile_rows;
            k = tn * gm::kSlotCols + 4 * (int)(i % kTileQuads);
            if (m >= M)
                continue;
        }
        float4 v;
        if (tile < t.full) {
            v = *reinterpret_cast<const float4 *>(a.acc + (int64_t)m * a.K + k);
        } else {
            const int64_t copy0 = (int64_t)(tile - t.full) * t.splits;
            const float *p = a.copies + (copy0 * a.bm + m % a.bm) * gm::kSlotCols + k % gm::kSlotCols;
            const int64_t stride = (int64_t)a.bm * gm::kSlotCols;
            v = *reinterpret_cast<const float4 *>(p);
#pragma unroll 4
            for (int s = 1; s < t.splits; ++s) {
                const float4 u = *reinterpret_cast<const float4 *>(p + s * stride);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
        }
        const int64_t row = a.rows != nullptr ? a.rows[m] : m;
        *reinterpret_cast<uint2 *>(a.dst + row * a.K + k) =
            make_uint2(to_bf16x2_bits(v.x, v.y), to_bf16x2_bits(v.z, v.w));
    }
}

inline cudaError_t launch_row_loss(const float *y, int64_t M, int64_t V, const int64_t *targets, int64_t ignore,
                                   float *loss, float *lse, cudaStream_t stream)
{
    return launch_dependent(row_loss_kernel, dim3(kRowCtas, (unsigned)M), kThreads, 0, stream, y, V, targets, ignore,
                            loss, lse);
}

inline cudaError_t launch_loss(const float2 *part, int64_t slices, int64_t M, const int64_t *targets, int64_t ignore,
                               int64_t V, const float *tlogit, float *loss, float *lse, cudaStream_t stream)
{
    return launch_dependent(loss_kernel, dim3((unsigned)((M + kThreads / 32 - 1) / (kThreads / 32))), kThreads, 0,
                            stream, part, slices, M, targets, ignore, V, tlogit, loss, lse);
}

inline cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream)
{
    return launch_dependent(compact_kernel, dim3((unsigned)((a.M + kCompactRows - 1) / kCompactRows)), kThreads, 0, stream, a);
}

inline cudaError_t launch_split_sum(const SumArgs &a, int num_sms, cudaStream_t stream)
{
    int64_t grid = ((int64_t)a.M * a.K / 4 + kThreads - 1) / kThreads;
    if (grid > 8 * (int64_t)num_sms)
        grid = 8 * (int64_t)num_sms;
    return launch_dependent(split_sum_kernel, dim3((unsigned)grid), kThreads, 0, stream, a);
}

}  // namespace ce
}  // namespace cr

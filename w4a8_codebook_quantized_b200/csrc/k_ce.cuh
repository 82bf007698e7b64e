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
constexpr int kSlice = 2048;  // columns per CTA of stats_kernel

using gm::join;

// Statistics of stored fp32 outputs y [M, V] (a decode batch, whose outputs
// the GEMV wrote), kSlice columns per CTA: grid (slices, M).
__global__ void __launch_bounds__(kThreads) stats_kernel(const float *__restrict__ y, int64_t V,
                                                         const int64_t *__restrict__ targets,
                                                         float2 *__restrict__ part, float *__restrict__ tlogit)
{
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float kNegInf = __int_as_float(0xFF800000);
    __shared__ float2 sh[kThreads / 32];
    const int64_t m = blockIdx.y, n0 = (int64_t)blockIdx.x * kSlice;
    const float *row = y + m * V;
    const int64_t t = targets[m];
    float v[kSlice / kThreads];
    float mx = kNegInf;
#pragma unroll
    for (int i = 0; i < kSlice / kThreads; ++i) {
        const int64_t n = n0 + i * kThreads + threadIdx.x;
        v[i] = n < V ? row[n] : kNegInf;
        if (n == t && n < V)
            tlogit[m] = v[i];
        mx = fmaxf(mx, v[i]);
    }
    float2 a = make_float2(__fmul_rn(mx, gm::kLog2e), 0.0f);
    const float base = a.x == kNegInf ? 0.0f : a.x;
#pragma unroll
    for (int i = 0; i < kSlice / kThreads; ++i)
        a.y += gm::ex2(__fmaf_rn(v[i], gm::kLog2e, -base));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        join(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, o), __shfl_xor_sync(0xFFFFFFFFu, a.y, o)));
    if ((threadIdx.x & 31) == 0)
        sh[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w)
            join(a, sh[w]);
        part[m * gridDim.x + blockIdx.x] = a;
    }
}

// lse and loss from the statistics, a warp per row: the lanes take every 32nd
// slice each and are joined in a fixed order.  The last steps are in fp64: a
// few operations per row, and the loss is often a small difference of larger
// numbers.
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
    if (lane == 0) {
        // the references are in units of the fp32 constant that made them
        const double l = (double)a.x / (double)gm::kLog2e + log((double)a.y);
        lse[m] = (float)l;
        const int64_t t = targets[m];
        float out = 0.0f;
        if (t != ignore)
            out = (t >= 0 && t < V) ? (float)(l - (double)tlogit[m]) : __int_as_float(0x7FC00000);
        loss[m] = out;
    }
}

// out[m, k] = bf16(sum over s of acc[s, m, k]), four elements per thread and
// step; the sums are taken in the order of s.
__global__ void __launch_bounds__(kThreads) sum_to_bf16_kernel(const float4 *__restrict__ acc, int splits,
                                                               int64_t split_stride4, int64_t n4,
                                                               uint2 *__restrict__ dst)
{
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n4; i += (int64_t)gridDim.x * kThreads) {
        float4 v = acc[i];
#pragma unroll 4
        for (int s = 1; s < splits; ++s) {
            const float4 u = acc[s * split_stride4 + i];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        dst[i] = make_uint2(to_bf16x2_bits(v.x, v.y), to_bf16x2_bits(v.z, v.w));
    }
}

inline cudaError_t launch_stats(const float *y, int64_t M, int64_t V, const int64_t *targets, float2 *part,
                                float *tlogit, cudaStream_t stream)
{
    return launch_dependent(stats_kernel, dim3((unsigned)((V + kSlice - 1) / kSlice), (unsigned)M), kThreads, 0,
                            stream, y, V, targets, part, tlogit);
}

inline cudaError_t launch_loss(const float2 *part, int64_t slices, int64_t M, const int64_t *targets, int64_t ignore,
                               int64_t V, const float *tlogit, float *loss, float *lse, cudaStream_t stream)
{
    return launch_dependent(loss_kernel, dim3((unsigned)((M + kThreads / 32 - 1) / (kThreads / 32))), kThreads, 0,
                            stream, part, slices, M, targets, ignore, V, tlogit, loss, lse);
}

// acc: `splits` blocks of split_rows x K fp32; dst [M, K] bf16.
inline cudaError_t launch_sum_to_bf16(const float *acc, int splits, int64_t split_rows, int64_t M, int64_t K,
                                      uint16_t *dst, int num_sms, cudaStream_t stream)
{
    const int64_t n4 = M * K / 4;
    int64_t grid = (n4 + kThreads - 1) / kThreads;
    if (grid > 8 * (int64_t)num_sms)
        grid = 8 * (int64_t)num_sms;
    return launch_dependent(sum_to_bf16_kernel, dim3((unsigned)grid), kThreads, 0, stream,
                            reinterpret_cast<const float4 *>(acc), splits, split_rows * K / 4, n4,
                            reinterpret_cast<uint2 *>(dst));
}

}  // namespace ce
}  // namespace cr

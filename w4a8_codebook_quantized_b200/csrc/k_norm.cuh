// k_norm.cuh -- what stands between two W4A8 layers: the root-mean-square norm
// with the residual's addition, fused with the block rotation and the
// per-token int8 quantisation of the next layer's input; its gradient; and the
// block rotation alone.
//
// Forward, per row (k_rotquant.cuh has the rotation's definition and fp32
// order, and the quantiser):
//   h  = bf16(x + residual)             (h = x without a residual)
//   rs = fp32(1 / sqrt(sum h^2 / K + eps))   sum, quotient and root in fp64
//   v  = (h * rs) * gamma               two fp32 operations
//   r  = v rotated block-wise;  xs = max |r| / qmax;  xq = clamp(rint(r / xs))
// The sum is taken in fp64: a square of a bf16 value is exact there, and the
// sum of a row keeps about 2^-50, so the fp32 result does not depend on the
// order of the additions and the whole row is bit-reproducible.
//
// Backward, per row, with dr the gradient of r (straight through the
// quantiser; the rotation is its own transpose and inverse):
//   dv = dr rotated;  xh = h * rs;  g = dv * gamma;  c = sum_k(g * xh) / K
//   dx = bf16(rs * (g - xh * c) [+ dres]);  dgamma[k] = sum_m dv * xh
// all in fp32.
//
// All three are bound by HBM: the forward's floor is 2 bytes in per element
// (4 with a residual) and 1 (3) out, the backward's 6 (8), the rotation's 4.
// Measured on B200 (copy bandwidth 6.5 TB/s), inputs larger than L2: forward
// 16384 x 8192 with a residual 167 us (5.6 TB/s), backward 8192 x 4096 with dres
// and dgamma 51 us (5.2 TB/s), rotation 4096 x 12288 37.5 us (5.4 TB/s).
#pragma once

#include <climits>
#include <initializer_list>

#include "cr_device.cuh"
#include "k_rotquant.cuh"

namespace cr {
namespace nm {

// ---------------------------------------------------------------- loads and sums

// Sixteen consecutive bf16 values as eight words (element 2i in the low half
// of word i).  Plain loads: the rows may be written earlier by this kernel.
// wide: every row starts on a 32-byte boundary, and one 256-bit access takes
// them: a warp's 32 lanes then cover whole lines, where two 128-bit accesses at
// a stride of 32 bytes each touch every line of the span (measured, 16384 x
// 8192 forward: 192 -> 168 us).
__device__ __forceinline__ void load16(const uint16_t *p, bool wide, uint32_t (&w)[8])
{
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p)
                     : "memory");
        return;
    }
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint4 b = *reinterpret_cast<const uint4 *>(p + 8);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

__device__ __forceinline__ void store16(uint16_t *p, bool wide, const uint32_t (&w)[8])
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
        return;
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Whether every given pointer starts on a 32-byte boundary (rows are multiples
// of 512 bytes; a null pointer counts as aligned).
inline bool all_wide(std::initializer_list<const void *> ps)
{
    uintptr_t bits = 0;
    for (const void *p : ps)
        bits |= reinterpret_cast<uintptr_t>(p);
    return (bits & 31) == 0;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// w = bf16(w + r), element-wise: one fp32 addition of the exact values,
// rounded once.
__device__ __forceinline__ void add16(uint32_t (&w)[8], const uint32_t (&r)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = to_bf16x2_bits(__fadd_rn(bf16_lo(w[i]), bf16_lo(r[i])), __fadd_rn(bf16_hi(w[i]), bf16_hi(r[i])));
}

// The magnitude of a bf16 value as a double, built from its bits (sign
// dropped, exponent rebias 127 -> 1023): two integer instructions instead of a
// conversion, which has a quarter of the rate.  Exact for normal values; zero
// and subnormals come out as at most 2^-126, whose square does not reach the
// 50th bit of a sum that has eps >= 1e-30 added.
__device__ __forceinline__ double mag_lo(uint32_t w)
{
    return __hiloint2double((int)(((w & 0x7FFFu) << 13) + 0x38000000u), 0);
}
__device__ __forceinline__ double mag_hi(uint32_t w)
{
    return __hiloint2double((int)(((w >> 3) & 0x0FFFE000u) + 0x38000000u), 0);
}

// Sum of the squares of sixteen bf16 values, two chains.
__device__ __forceinline__ double squares16(const uint32_t (&w)[8])
{
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double a = mag_lo(w[i]), b = mag_hi(w[i]);
        s0 = __fma_rn(a, a, s0);
        s1 = __fma_rn(b, b, s1);
    }
    return s0 + s1;
}

// rs of the row, from every thread's share of the sum of squares: the warps'
// sums in shared memory, then every thread adds them in the same order and
// takes the root (some twenty fp64 instructions a warp; one warp doing it for
// all costs a second barrier).
template <int THREADS>
__device__ __forceinline__ float row_rs(double ss, double inv_k, double eps, double *warp_ss)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if ((threadIdx.x & 31) == 0)
        warp_ss[threadIdx.x >> 5] = ss;
    __syncthreads();
    double t[THREADS / 32];
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w)
        t[w] = warp_ss[w];
    double sum = t[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w)
        sum += t[w];
    return (float)rsqrt(fma(sum, inv_k, eps));
}

// Sixteen consecutive weights as fp32 (GBF16: stored as bf16).
template <bool GBF16>
__device__ __forceinline__ void load_gamma16(const void *gamma, int64_t k, float (&g)[16])
{
    if constexpr (GBF16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(gamma) + k);
        const uint4 a = __ldg(p), b = __ldg(p + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[2 * i] = bf16_lo(w[i]);
            g[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(gamma) + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 a = __ldg(p + i);
            g[4 * i] = a.x, g[4 * i + 1] = a.y, g[4 * i + 2] = a.z, g[4 * i + 3] = a.w;
        }
    }
}

// The same as eight fp32 pairs.
template <bool GBF16>
__device__ __forceinline__ void load_gamma_pairs(const void *gamma, int64_t k, uint64_t (&g)[8])
{
    float f[16];
    load_gamma16<GBF16>(gamma, k, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        g[i] = pack2(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
}

// Both bf16 values of a word as an fp32 pair.
__device__ __forceinline__ uint64_t pair_of(uint32_t w) { return pack2(w << 16, w & 0xFFFF0000u); }

// The maximum over the CTA of a non-negative, NaN-free value.
template <int THREADS>
__device__ __forceinline__ float block_max(float amax, float *warp_max)
{
    uint32_t bits = __float_as_uint(amax);
    asm volatile("redux.sync.max.u32 %0, %0, 0xffffffff;" : "+r"(bits));
    if ((threadIdx.x & 31) == 0)
        warp_max[threadIdx.x >> 5] = __uint_as_float(bits);
    __syncthreads();
    float m = warp_max[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w)
        m = fmaxf(m, warp_max[w]);
    return m;
}

// The row's scale and what the quantiser needs of it, from max |R| = 16 max |r|
// (k_rotquant.cuh).
struct RowScale {
    float scale, inv16;
    bool exact_row;
    __device__ __forceinline__ RowScale(float rmax, int qmax)
    {
        const float rowmax = __fmul_rn(rmax, 0.0625f);
        scale = (rowmax > 0.0f) ? __fdiv_rn(rowmax, (float)qmax) : 1.0f;
        exact_row = rowmax > 0.0f && rowmax < 7.8886091e-31f;  // max |r| < 2^-100
        inv16 = __fmul_rn(__frcp_rn(scale), 0.0625f);
    }
};

struct FwdArgs {
    const uint16_t *x, *res;
    const void *gamma;
    double eps, inv_k;
    int64_t M, K;
    int qmax;
    bool wide;      // x, res and h on 32-byte boundaries
    uint16_t *h;
    int8_t *xq;
    float *xs, *rs;
};

// Rows m >= M of the decode GEMV's padded operand: zeros with scale 1.
__device__ __forceinline__ bool padding_row(const FwdArgs &a, int64_t m)
{
    if (m < a.M)
        return false;
    for (int64_t c = threadIdx.x; c < a.K / 16; c += blockDim.x)
        reinterpret_cast<uint4 *>(a.xq + m * a.K)[c] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0)
        a.xs[m] = 1.0f;
    return true;
}

// ---------------------------------------------------------------- forward, short batches
//
// One CTA per row and one 256-element block per half-warp, as
// rotquant_rows_kernel: few CTAs run, and the chain of dependent steps is what
// a decode step waits for.  J blocks per half-warp stay in registers from the
// load to the store; kRecompute (longer rows) reads h back for each of its two
// passes after the sum.
template <int J, bool kRecompute, int THREADS, bool GBF16>
__global__ void __launch_bounds__(THREADS) rmsnorm_rows_kernel(const FwdArgs a)
{
    constexpr int kHalfWarps = THREADS / 16;
    __shared__ __align__(16) float tr_all[kHalfWarps][16 * 16 + 16];
    __shared__ __align__(16) uint8_t tb_all[kHalfWarps][272];
    __shared__ double warp_ss[THREADS / 32];
    __shared__ float warp_max[THREADS / 32];

    asm volatile("griddepcontrol.launch_dependents;" :::);
    if (threadIdx.x == 0 && (int64_t)blockIdx.x < a.M) {
        bulk_prefetch_l2(a.x + (int64_t)blockIdx.x * a.K, (uint32_t)(a.K * 2));
        if (a.res != nullptr)
            bulk_prefetch_l2(a.res + (int64_t)blockIdx.x * a.K, (uint32_t)(a.K * 2));
    }
    // nothing is read or written before the previous kernel has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int64_t m = blockIdx.x;
    if (padding_row(a, m))
        return;
    const int tid = threadIdx.x, hw = tid >> 4, L = tid & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1));
    const int NB = (int)(a.K / 256);
    const uint16_t *xrow = a.x + m * a.K;
    const uint16_t *rrow = a.res != nullptr ? a.res + m * a.K : nullptr;
    uint16_t *hrow = a.h + m * a.K;
    int8_t *qrow = a.xq + m * a.K;
    float *tr = tr_all[hw];
    uint8_t *tb = tb_all[hw];

    constexpr int kHeld = kRecompute ? 1 : J;
    uint32_t w[kHeld][8];
    double ss = 0.0;
    auto load_h = [&](int b, uint32_t (&wj)[8]) {
        load16(xrow + 256 * b + 16 * L, a.wide, wj);
        if (rrow != nullptr) {
            uint32_t r[8];
            load16(rrow + 256 * b + 16 * L, a.wide, r);
            add16(wj, r);
            store16(hrow + 256 * b + 16 * L, a.wide, wj);
        }
        ss += squares16(wj);
    };
    if constexpr (!kRecompute) {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (hw + kHalfWarps * j < NB)
                load_h(hw + kHalfWarps * j, w[j]);
    } else {
        for (int b = hw; b < NB; b += kHalfWarps)
            load_h(b, w[0]);
    }
    const float rs = row_rs<THREADS>(ss, a.inv_k, a.eps, warp_ss);

    float v[kHeld][16];
    auto rotate = [&](int b, const uint32_t (&wj)[8], float (&vj)[16]) {
        float g[16];
        load_gamma16<GBF16>(a.gamma, 256 * b + 16 * L, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            vj[2 * i] = __fmul_rn(__fmul_rn(bf16_lo(wj[i]), rs), g[2 * i]);
            vj[2 * i + 1] = __fmul_rn(__fmul_rn(bf16_hi(wj[i]), rs), g[2 * i + 1]);
        }
        rq::rotate_regs(L, tr, hmask, vj);
    };
    const uint16_t *again = rrow != nullptr ? hrow : xrow;  // where this thread finds its values of h again
    float amax = 0.0f;
    if constexpr (!kRecompute) {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (hw + kHalfWarps * j < NB) {
                rotate(hw + kHalfWarps * j, w[j], v[j]);
                amax = fmaxf(amax, rq::max_abs16(v[j]));
            }
    } else {
        for (int b = hw; b < NB; b += kHalfWarps) {
            load16(again + 256 * b + 16 * L, a.wide, w[0]);
            rotate(b, w[0], v[0]);
            amax = fmaxf(amax, rq::max_abs16(v[0]));
        }
    }
    const RowScale s(block_max<THREADS>(amax, warp_max), a.qmax);
    if constexpr (!kRecompute) {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (hw + kHalfWarps * j < NB)
                rq::quantise_store(v[j], s.scale, s.inv16, a.qmax, s.exact_row, L, tb, hmask,
                                   qrow + 256 * (hw + kHalfWarps * j));
    } else {
        for (int b = hw; b < NB; b += kHalfWarps) {
            load16(again + 256 * b + 16 * L, a.wide, w[0]);
            rotate(b, w[0], v[0]);
            rq::quantise_store(v[0], s.scale, s.inv16, a.qmax, s.exact_row, L, tb, hmask, qrow + 256 * b);
        }
    }
    if (tid == 0) {
        a.xs[m] = s.scale;
        if (a.rs != nullptr)
            a.rs[m] = rs;
    }
}

// ---------------------------------------------------------------- forward, many rows
//
// A half-warp owns a pair of blocks and works on both in packed fp32x2
// arithmetic (each half rounded as the scalar instruction rounds it), as
// rotquant_pairs_kernel: at these sizes the scalar form is bound by the
// instructions it issues.
// (Three CTAs of 384 threads an SM take 56 registers, two fewer than it has by
// itself.)
template <int J, bool kRecompute, int THREADS, bool GBF16>
__global__ void __launch_bounds__(THREADS, THREADS == 384 ? 3 : 0) rmsnorm_pairs_kernel(const FwdArgs a)
{
    constexpr int kHalfWarps = THREADS / 16;
    extern __shared__ __align__(16) uint64_t nm_smem[];
    __shared__ double warp_ss[THREADS / 32];
    __shared__ float warp_max[THREADS / 32];

    asm volatile("griddepcontrol.launch_dependents;" :::);
    if (threadIdx.x == 0 && (int64_t)blockIdx.x < a.M) {
        bulk_prefetch_l2(a.x + (int64_t)blockIdx.x * a.K, (uint32_t)(a.K * 2));
        if (a.res != nullptr)
            bulk_prefetch_l2(a.res + (int64_t)blockIdx.x * a.K, (uint32_t)(a.K * 2));
    }
    // nothing is read or written before the previous kernel has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int64_t m = blockIdx.x;
    if (padding_row(a, m))
        return;
    const int tid = threadIdx.x, hw = tid >> 4, L = tid & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1));
    const int NB = (int)(a.K / 256);
    const int NP = (NB + 1) / 2;  // block pairs (2p, 2p + 1); the last one may be alone
    const uint16_t *xrow = a.x + m * a.K;
    const uint16_t *rrow = a.res != nullptr ? a.res + m * a.K : nullptr;
    uint16_t *hrow = a.h + m * a.K;
    int8_t *qrow = a.xq + m * a.K;
    uint64_t *tr = nm_smem + 256 * hw;
    uint8_t *tb = reinterpret_cast<uint8_t *>(tr) + 64 * (hw & 1);

    constexpr int kHeld = kRecompute ? 1 : J;
    uint32_t w0[kHeld][8], w1[kHeld][8];
    double ss = 0.0;
    auto load_h = [&](int p, uint32_t (&u0)[8], uint32_t (&u1)[8]) {
        const int64_t k0 = 512 * (int64_t)p + 16 * L;
        const bool two = 2 * p + 1 < NB;
        load16(xrow + k0, a.wide, u0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u1[i] = 0u;
        if (two)
            load16(xrow + k0 + 256, a.wide, u1);
        if (rrow != nullptr) {
            uint32_t r0[8], r1[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            load16(rrow + k0, a.wide, r0);
            if (two)
                load16(rrow + k0 + 256, a.wide, r1);
            add16(u0, r0);
            add16(u1, r1);
            store16(hrow + k0, a.wide, u0);
            if (two)
                store16(hrow + k0 + 256, a.wide, u1);
        }
        ss += squares16(u0);
        if (two)
            ss += squares16(u1);
    };
    if constexpr (!kRecompute) {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (hw + kHalfWarps * j < NP)
                load_h(hw + kHalfWarps * j, w0[j], w1[j]);
    } else {
        for (int p = hw; p < NP; p += kHalfWarps)
            load_h(p, w0[0], w1[0]);
    }
    const float rs = row_rs<THREADS>(ss, a.inv_k, a.eps, warp_ss);
    const uint64_t rs2 = pack2(__float_as_uint(rs), __float_as_uint(rs));

    uint64_t v[kHeld][16];
    auto rotate = [&](int p, const uint32_t (&u0)[8], const uint32_t (&u1)[8], uint64_t (&vj)[16]) {
        float g0[16], g1[16];
        const int64_t k0 = 512 * (int64_t)p + 16 * L;
        load_gamma16<GBF16>(a.gamma, k0, g0);
        if (2 * p + 1 < NB) {
            load_gamma16<GBF16>(a.gamma, k0 + 256, g1);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                g1[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t lo = pack2(u0[i] << 16, u1[i] << 16);
            const uint64_t hi = pack2(u0[i] & 0xFFFF0000u, u1[i] & 0xFFFF0000u);
            vj[2 * i] = mul2(mul2(lo, rs2), pack2(__float_as_uint(g0[2 * i]), __float_as_uint(g1[2 * i])));
            vj[2 * i + 1] = mul2(mul2(hi, rs2),
                                     pack2(__float_as_uint(g0[2 * i + 1]), __float_as_uint(g1[2 * i + 1])));
        }
        rq::rotate_pair_regs(L, tr, hmask, vj);
    };
    auto reload = [&](int p) {  // this thread's values of h again
        const uint16_t *src = (rrow != nullptr ? hrow : xrow) + 512 * (int64_t)p + 16 * L;
        load16(src, a.wide, w0[0]);
        if (2 * p + 1 < NB)
            load16(src + 256, a.wide, w1[0]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w1[0][i] = 0u;
    };
    auto dst1 = [&](int p) { return 2 * p + 1 < NB ? qrow + 256 * (2 * p + 1) : nullptr; };
    float amax = 0.0f;
    if constexpr (!kRecompute) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int p = hw + kHalfWarps * j;
            if (p < NP) {
                rotate(p, w0[j], w1[j], v[j]);
                amax = fmaxf(amax, rq::max_abs_pairs(v[j]));
            }
        }
    } else {
        for (int p = hw; p < NP; p += kHalfWarps) {
            reload(p);
            rotate(p, w0[0], w1[0], v[0]);
            amax = fmaxf(amax, rq::max_abs_pairs(v[0]));
        }
    }
    const RowScale s(block_max<THREADS>(amax, warp_max), a.qmax);
    if constexpr (!kRecompute) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int p = hw + kHalfWarps * j;
            if (p < NP)
                rq::quantise_store_pair(v[j], s.scale, s.inv16, a.qmax, s.exact_row, L, tb, hmask, qrow + 512 * p,
                                        dst1(p));
        }
    } else {
        for (int p = hw; p < NP; p += kHalfWarps) {
            reload(p);
            rotate(p, w0[0], w1[0], v[0]);
            rq::quantise_store_pair(v[0], s.scale, s.inv16, a.qmax, s.exact_row, L, tb, hmask, qrow + 512 * p,
                                    dst1(p));
        }
    }
    if (tid == 0) {
        a.xs[m] = s.scale;
        if (a.rs != nullptr)
            a.rs[m] = rs;
    }
}

// ---------------------------------------------------------------- forward, many short rows
//
// K <= 1536: G half-warps per row (1 for K <= 512, 2 for K <= 1024, 3 above), a
// pair of blocks each, eight half-warps a CTA (six for G = 3).  With G <= 2 a
// row is one warp's or half a warp's, so its two reductions are shuffles and no
// CTA-wide barrier is left.  With a CTA per row three quarters of its threads
// had no block at K = 256 (393216 rows: 765 us instead of 184), and one in four
// at K = 1536 (65536 rows: 146 us instead of 138).  Eight CTAs an SM asked for
// (64 registers) take G = 1 from 196 to 184 us; G = 2 has 64 by itself and was
// 2 % slower when asked.
constexpr int small_half_warps(int G) { return G == 3 ? 6 : 8; }

template <int G, bool GBF16>
__global__ void __launch_bounds__(16 * small_half_warps(G), G == 1 ? 8 : 0) rmsnorm_small_kernel(const FwdArgs a, int64_t MP)
{
    constexpr int kHalfWarps = small_half_warps(G);
    __shared__ __align__(16) uint64_t tr_all[kHalfWarps][256];
    __shared__ double hw_ss[kHalfWarps];  // G = 3: a row's shares
    __shared__ float hw_max[kHalfWarps];
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, hw = tid >> 4, L = tid & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1)), rmask = G == 2 ? 0xFFFFFFFFu : hmask;
    const int64_t m = (kHalfWarps / G) * (int64_t)blockIdx.x + hw / G;
    const int p = hw % G;  // the half-warp's pair of blocks
    const int NB = (int)(a.K / 256);
    if (m >= MP)
        return;
    if (m >= a.M) {  // padding row of the decode GEMV's operand
        for (int64_t c = 16 * p + L; c < a.K / 16; c += 16 * G)
            reinterpret_cast<uint4 *>(a.xq + m * a.K)[c] = make_uint4(0u, 0u, 0u, 0u);
        if (p == 0 && L == 0)
            a.xs[m] = 1.0f;
        return;
    }
    const bool one = 2 * p < NB, two = 2 * p + 1 < NB;
    const int64_t at = m * a.K + 512 * p + 16 * L;
    uint64_t *tr = tr_all[hw];
    uint8_t *tb = reinterpret_cast<uint8_t *>(tr) + 64 * (hw & 1);
    uint32_t w0[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, w1[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    double ss = 0.0;
    auto load_h = [&](int64_t k, uint32_t (&w)[8]) {
        load16(a.x + k, a.wide, w);
        if (a.res != nullptr) {
            uint32_t r[8];
            load16(a.res + k, a.wide, r);
            add16(w, r);
            store16(a.h + k, a.wide, w);
        }
        ss += squares16(w);
    };
    if (one)
        load_h(at, w0);
    if (two)
        load_h(at + 256, w1);
#pragma unroll
    for (int o = G == 2 ? 16 : 8; o >= 1; o >>= 1)
        ss += __shfl_xor_sync(rmask, ss, o);
    if constexpr (G == 3) {  // (rows without work have left; the barriers wait for the others only)
        if (L == 0)
            hw_ss[hw] = ss;
        __syncthreads();
        ss = (hw_ss[hw - p] + hw_ss[hw - p + 1]) + hw_ss[hw - p + 2];
    }
    const float rs = (float)rsqrt(fma(ss, a.inv_k, a.eps));
    const uint64_t rs2 = pair_both(rs);
    float g0[16], g1[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        g0[i] = g1[i] = 0.0f;
    if (one)
        load_gamma16<GBF16>(a.gamma, 512 * p + 16 * L, g0);
    if (two)
        load_gamma16<GBF16>(a.gamma, 512 * p + 256 + 16 * L, g1);
    uint64_t v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = mul2(mul2(pack2(w0[i] << 16, w1[i] << 16), rs2),
                        pack2(__float_as_uint(g0[2 * i]), __float_as_uint(g1[2 * i])));
        v[2 * i + 1] = mul2(mul2(pack2(w0[i] & 0xFFFF0000u, w1[i] & 0xFFFF0000u), rs2),
                            pack2(__float_as_uint(g0[2 * i + 1]), __float_as_uint(g1[2 * i + 1])));
    }
    rq::rotate_pair_regs(L, tr, hmask, v);
    float rmax = __uint_as_float(__reduce_max_sync(rmask, __float_as_uint(rq::max_abs_pairs(v))));
    if constexpr (G == 3) {
        if (L == 0)
            hw_max[hw] = rmax;
        __syncthreads();
        rmax = fmaxf(fmaxf(hw_max[hw - p], hw_max[hw - p + 1]), hw_max[hw - p + 2]);
    }
    const RowScale s(rmax, a.qmax);
    if (one)
        rq::quantise_store_pair(v, s.scale, s.inv16, a.qmax, s.exact_row, L, tb, hmask, a.xq + m * a.K + 512 * p,
                                two ? a.xq + m * a.K + 512 * p + 256 : nullptr);
    if (p == 0 && L == 0) {
        a.xs[m] = s.scale;
        if (a.rs != nullptr)
            a.rs[m] = rs;
    }
}

template <bool GBF16, int THREADS>
inline cudaError_t launch_fwd_rows(const FwdArgs &a, int64_t MP, cudaStream_t stream)
{
    constexpr int kHalfWarps = THREADS / 16;
    const int64_t per_hw = (a.K / 256 + kHalfWarps - 1) / kHalfWarps;  // blocks per half-warp
    void (*kern)(FwdArgs) = per_hw <= 1   ? rmsnorm_rows_kernel<1, false, THREADS, GBF16>
                            : per_hw == 2 ? rmsnorm_rows_kernel<2, false, THREADS, GBF16>
                                          : rmsnorm_rows_kernel<1, true, THREADS, GBF16>;
    return launch_dependent(kern, dim3((unsigned)(MP)), THREADS, 0, stream, a);
}

// Opt the 384- to 1024-thread CTAs of the packed form into their transpose
// buffers (above 48 KB).  Once per device, before the first launch.
inline cudaError_t set_attributes()
{
    struct Need {
        void (*f)(FwdArgs);
        int bytes;
    };
    const Need need[] = {
        {rmsnorm_pairs_kernel<1, false, 1024, true>, rq::smem_bytes<1024>()},
        {rmsnorm_pairs_kernel<1, false, 1024, false>, rq::smem_bytes<1024>()},
        {rmsnorm_pairs_kernel<1, false, 512, true>, rq::smem_bytes<512>()},
        {rmsnorm_pairs_kernel<1, false, 512, false>, rq::smem_bytes<512>()},
        {rmsnorm_pairs_kernel<1, false, 448, true>, rq::smem_bytes<448>()},
        {rmsnorm_pairs_kernel<1, false, 448, false>, rq::smem_bytes<448>()},
        {rmsnorm_pairs_kernel<1, true, 512, true>, rq::smem_bytes<512>()},
        {rmsnorm_pairs_kernel<1, true, 512, false>, rq::smem_bytes<512>()},
        {rmsnorm_pairs_kernel<1, false, 384, true>, rq::smem_bytes<384>()},
        {rmsnorm_pairs_kernel<1, false, 384, false>, rq::smem_bytes<384>()},
    };
    for (const Need &n : need) {
        const cudaError_t e = cudaFuncSetAttribute(n.f, cudaFuncAttributeMaxDynamicSharedMemorySize, n.bytes);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

template <bool GBF16>
inline cudaError_t launch_fwd_t(const FwdArgs &a, int64_t MP, cudaStream_t stream)
{
    if (MP <= rq::kShortRows)
        return a.K >= 8192 ? launch_fwd_rows<GBF16, 512>(a, MP, stream) : launch_fwd_rows<GBF16, 256>(a, MP, stream);
    auto several = [&](auto half_warps) {
        constexpr int G = decltype(half_warps)::value, rows = small_half_warps(G) / G;
        return launch_dependent(rmsnorm_small_kernel<G, GBF16>, dim3((unsigned)((MP + rows - 1) / rows)),
                                16 * small_half_warps(G), 0, stream, a, MP);
    };
    auto in_one = [&](auto threads) {  // a half-warp per pair of blocks
        constexpr int T = decltype(threads)::value;
        return launch_dependent(rmsnorm_pairs_kernel<1, false, T, GBF16>, dim3((unsigned)MP), T, rq::smem_bytes<T>(),
                                stream, a);
    };
    const int64_t pairs = (a.K / 256 + 1) / 2;
    if (pairs == 1)
        return several(std::integral_constant<int, 1>{});
    if (pairs == 2)
        return several(std::integral_constant<int, 2>{});
    if (pairs == 3)
        return several(std::integral_constant<int, 3>{});
    if (pairs <= 4)
        return in_one(std::integral_constant<int, 64>{});
    if (pairs <= 6)
        return in_one(std::integral_constant<int, 96>{});
    if (pairs <= 8)
        return in_one(std::integral_constant<int, 128>{});
    if (pairs <= 10)
        return in_one(std::integral_constant<int, 160>{});
    if (pairs <= 12)
        return in_one(std::integral_constant<int, 192>{});
    if (pairs <= 14)
        return in_one(std::integral_constant<int, 224>{});
    if (pairs <= 16)
        return in_one(std::integral_constant<int, 256>{});
    if (pairs <= 20)
        return in_one(std::integral_constant<int, 320>{});
    if (pairs <= 24)
        return in_one(std::integral_constant<int, 384>{});
    if (pairs <= 28)
        return in_one(std::integral_constant<int, 448>{});
    if (pairs <= 32)
        return in_one(std::integral_constant<int, 512>{});
    if (pairs <= 64)
        return in_one(std::integral_constant<int, 1024>{});
    return launch_dependent(rmsnorm_pairs_kernel<1, true, 512, GBF16>, dim3((unsigned)(MP)), 512, rq::smem_bytes<512>(), stream, a);
}

// Short batches take the scalar form, 512 threads for K >= 8192 and 256 below;
// longer ones the packed form: several rows a CTA up to K = 1536, then one
// half-warp per block pair while that fits a CTA (K <= 32768), and the
// re-reading form beyond.  At 64 registers an SM holds 1024 threads, so a CTA
// has as few as the row's pairs take (19660 x 5120: 148 us with 256 threads,
// 122 with 160; 9144 x 11008: 164 us with two CTAs of 384, 139 with three).
inline cudaError_t launch_fwd(FwdArgs a, int64_t MP, bool gamma_bf16, cudaStream_t stream)
{
    a.inv_k = 1.0 / (double)a.K;
    a.wide = all_wide({a.x, a.res, a.h});
    return gamma_bf16 ? launch_fwd_t<true>(a, MP, stream) : launch_fwd_t<false>(a, MP, stream);
}

// ---------------------------------------------------------------- the rotation back in row order

// Rotate one block held in row order, v[i] = elements 16L + 2i (low half) and
// 16L + 2i + 1, and return 16 times the result in row order.  The digits whose
// stride is a multiple of 4 places work on both elements of a pair at once.
// Two transposes through `tr`: chunk c of row a lives at chunk position
// c ^ ((a >> 1) & 3), which makes the 16-byte and the scalar side conflict-free.
__device__ __forceinline__ void rotate_rows16(int L, float *tr, unsigned hmask, uint64_t (&v)[8])
{
    auto digits = [](uint64_t (&u)[8]) {  // stride 1, then stride 4, of the places 0..15
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t a0, a1, a2, a3;
            unpack2(u[2 * q], a0, a1);
            unpack2(u[2 * q + 1], a2, a3);
            float f0 = __uint_as_float(a0), f1 = __uint_as_float(a1), f2 = __uint_as_float(a2),
                  f3 = __uint_as_float(a3);
            rq::h4_quad(f0, f1, f2, f3);
            u[2 * q] = pack2(__float_as_uint(f0), __float_as_uint(f1));
            u[2 * q + 1] = pack2(__float_as_uint(f2), __float_as_uint(f3));
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            rq::h4_quad2(u[q], u[q + 2], u[q + 4], u[q + 6]);
    };
    digits(v);
    uint4 *rowp = reinterpret_cast<uint4 *>(tr + 16 * L);
    const int sw = (L >> 1) & 3;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t a0, a1, b0, b1;
        unpack2(v[2 * c], a0, a1);
        unpack2(v[2 * c + 1], b0, b1);
        rowp[c ^ sw] = make_uint4(a0, a1, b0, b1);
    }
    __syncwarp(hmask);
    uint32_t *col[4];  // this lane's column in rows whose (a >> 1) & 3 is k
#pragma unroll
    for (int k = 0; k < 4; ++k)
        col[k] = reinterpret_cast<uint32_t *>(tr) + 4 * ((L >> 2) ^ k) + (L & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = pack2(col[i & 3][32 * i], col[i & 3][32 * i + 16]);
    digits(v);
    // a lane's column is its own: it goes back to the places it came from
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t lo, hi;
        unpack2(v[i], lo, hi);
        col[i & 3][32 * i] = lo;
        col[i & 3][32 * i + 16] = hi;
    }
    __syncwarp(hmask);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 t = rowp[c ^ sw];
        v[2 * c] = pack2(t.x, t.y);
        v[2 * c + 1] = pack2(t.z, t.w);
    }
    __syncwarp(hmask);
}

// out = bf16(x rotated): a half-warp per pair of blocks, counted over all rows
// (the loop is for more than fit one grid), in the packed arithmetic of the
// many-row forward.  On the way back the two blocks' values of a place share a
// word, so that transpose moves half the bytes of an fp32 one; the row's words
// are then taken apart by byte permutes.  out may be x: a block is read and
// written by the same half-warp.
constexpr int kRotThreads = 256;

__global__ void __launch_bounds__(kRotThreads, 4) rotate_kernel(const uint16_t *x, int64_t blocks, uint16_t *out,
                                                               bool wide)
{
    __shared__ __align__(16) uint64_t tr_all[kRotThreads / 16][16 * 16];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hw = threadIdx.x >> 4, L = threadIdx.x & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1));
    uint64_t *tr = tr_all[hw];
    // 64 bytes in for the odd half-warp: the word stores of a warp's two halves
    // fall in different banks
    uint32_t *tw = reinterpret_cast<uint32_t *>(tr) + 16 * (hw & 1);
    for (int64_t p = (int64_t)blockIdx.x * (kRotThreads / 16) + hw; 2 * p < blocks;
         p += (int64_t)gridDim.x * (kRotThreads / 16)) {
        const bool two = 2 * p + 1 < blocks;
        uint32_t w0[8], w1[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        load16(x + 512 * p + 16 * L, wide, w0);
        if (two)
            load16(x + 512 * p + 256 + 16 * L, wide, w1);
        uint64_t v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = pack2(w0[i] << 16, w1[i] << 16);
            v[2 * i + 1] = pack2(w0[i] & 0xFFFF0000u, w1[i] & 0xFFFF0000u);
        }
        rq::rotate_pair_regs(L, tr, hmask, v);
        // column L out: word (a, L) at chunk (L / 4) ^ ((a / 2) % 4) of row a
#pragma unroll
        for (int a = 0; a < 16; ++a) {
            uint32_t lo, hi;
            unpack2(mul2(v[a], 0x3D8000003D800000ull), lo, hi);  // times 1/16
            tw[16 * a + 4 * ((L >> 2) ^ ((a >> 1) & 3)) + (L & 3)] =
                to_bf16x2_bits(__uint_as_float(lo), __uint_as_float(hi));
        }
        __syncwarp(hmask);
        const uint4 *rowp = reinterpret_cast<const uint4 *>(tw + 16 * L);
        const int sw = (L >> 1) & 3;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 t = rowp[c ^ sw];
            w0[2 * c] = prmt(t.x, t.y, 0x5410u);
            w1[2 * c] = prmt(t.x, t.y, 0x7632u);
            w0[2 * c + 1] = prmt(t.z, t.w, 0x5410u);
            w1[2 * c + 1] = prmt(t.z, t.w, 0x7632u);
        }
        __syncwarp(hmask);
        store16(out + 512 * p + 16 * L, wide, w0);
        if (two)
            store16(out + 512 * p + 256 + 16 * L, wide, w1);
    }
}

inline cudaError_t launch_rotate(const uint16_t *x, int64_t M, int64_t K, uint16_t *out, cudaStream_t stream)
{
    const int64_t blocks = M * (K / 256);
    int64_t grid = (blocks + kRotThreads / 8 - 1) / (kRotThreads / 8);
    if (grid > INT_MAX)
        grid = INT_MAX;
    return launch_dependent(rotate_kernel, dim3((unsigned)(grid)), kRotThreads, 0, stream, x, blocks, out, all_wide({x, out}));
}

// ---------------------------------------------------------------- backward
//
// A persistent grid over rows, so that a CTA adds up its share of dgamma in
// registers (one value per element of its blocks) and writes it once, as a row
// of the partials [P, K]; a second kernel adds the partials in a fixed order, so
// dgamma is the same from run to run.
struct BwdArgs {
    const uint16_t *dr, *h;
    const void *gamma;
    const float *rs;
    const uint16_t *dres;
    int64_t M, K;
    uint16_t *dx;
    float *part;  // [P, K], or null: no dgamma
    bool wide;    // dr, h, dres and dx on 32-byte boundaries
};

// Sum over the CTA; `slot` alternates between two rows of warp sums, so one
// barrier per call is enough.
template <int THREADS>
__device__ __forceinline__ float block_sum(float s, float (*warp_sum)[THREADS / 32], int slot)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 31) == 0)
        warp_sum[slot][threadIdx.x >> 5] = s;
    __syncthreads();
    float t = warp_sum[slot][0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w)
        t += warp_sum[slot][w];
    return t;
}

// What the backward kernels share: one block's arithmetic in packed pairs of
// neighbouring elements.  V = 16 dv comes out of the rotation; the 1/16 (exact)
// sits in rs16 = rs / 16: with
//   g' = V * gamma,  xh' = h * rs16:  V * xh' = dv * xh,  g' * xh' = g * xh,
//   dx = (g' - h * (16 c rs)) * rs16 + dres.
// (No rs * rs, which leaves fp32 for rows above 1e19; where 16 c rs is subnormal
// its lost bits change dx by less than 2^-140.)
struct BwdBlock {
    uint32_t d[8], h[8], r[8];  // dr, h and dres of the block's sixteen elements

    __device__ __forceinline__ void load(const BwdArgs &a, int64_t at)
    {
        load16(a.dr + at, a.wide, d);
        load16(a.h + at, a.wide, h);
        if (a.dres != nullptr) {
            load16(a.dres + at, a.wide, r);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = 0u;
        }
    }
    // g' of the block; adds dv * xh to acc and g * xh to s
    template <bool GBF16>
    __device__ __forceinline__ void first(const BwdArgs &a, int64_t k, int L, float *tr, unsigned hmask, uint64_t rs16,
                                          uint64_t (&g)[8], uint64_t (&acc)[8], uint64_t &s) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            g[i] = pair_of(d[i]);
        rotate_rows16(L, tr, hmask, g);
        uint64_t gm[8];
        load_gamma_pairs<GBF16>(a.gamma, k, gm);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t xh = mul2(pair_of(h[i]), rs16);
            acc[i] = fma2(g[i], xh, acc[i]);
            g[i] = mul2(g[i], gm[i]);
            s = fma2(g[i], xh, s);
        }
    }
    __device__ __forceinline__ void finish(const BwdArgs &a, int64_t at, const uint64_t (&g)[8], float rs, float c) const
    {
        const uint64_t rs16 = pair_both(rs * 0.0625f), k = pair_both(-16.0f * c * rs);
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo, hi;
            unpack2(fma2(fma2(pair_of(h[i]), k, g[i]), rs16, pair_of(r[i])), lo, hi);
            o[i] = to_bf16x2_bits(__uint_as_float(lo), __uint_as_float(hi));
        }
        store16(a.dx + at, a.wide, o);
    }
};

__device__ __forceinline__ float sum_pair(uint64_t v)
{
    uint32_t lo, hi;
    unpack2(v, lo, hi);
    return __uint_as_float(lo) + __uint_as_float(hi);
}

__device__ __forceinline__ void store_partial(float *p, const uint64_t (&acc)[8])
{
    ulonglong2 *pp = reinterpret_cast<ulonglong2 *>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        pp[q] = make_ulonglong2(acc[2 * q], acc[2 * q + 1]);
}

// K <= 512: a row is half a warp's (K = 256) or a warp's, 8 / G rows at once in
// a CTA of eight half-warps, the row's sum a few shuffles; a CTA adds up its
// row groups' shares of dgamma in shared memory at the end.
template <int G, bool GBF16>
__global__ void __launch_bounds__(128) rmsnorm_backward_small_kernel(const BwdArgs a)
{
    __shared__ __align__(16) float tr_all[8][16 * 16 + 16];
    __shared__ __align__(16) float share[8][256];  // written in 16-byte words (store_partial)
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hw = threadIdx.x >> 4, L = threadIdx.x & 15, b = hw % G;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1)), rmask = G == 1 ? hmask : 0xFFFFFFFFu;
    const float inv_k = 1.0f / (float)a.K;
    const int64_t k = 256 * b + 16 * L, step = (8 / G) * (int64_t)gridDim.x;
    uint64_t acc[8] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
    int64_t m = (8 / G) * (int64_t)blockIdx.x + hw / G;
    BwdBlock next;
    float nrs = 0.0f;
    if (m < a.M) {
        next.load(a, m * a.K + k);
        nrs = a.rs[m];
    }
    for (; m < a.M; m += step) {
        const BwdBlock cur = next;
        const float rs = nrs;
        if (m + step < a.M) {
            next.load(a, (m + step) * a.K + k);
            nrs = a.rs[m + step];
        }
        uint64_t g[8], s2 = 0ull;
        cur.first<GBF16>(a, k, L, tr_all[hw], hmask, pair_both(rs * 0.0625f), g, acc, s2);
        float s = sum_pair(s2);
#pragma unroll
        for (int o = 8 * G; o >= 1; o >>= 1)
            s += __shfl_xor_sync(rmask, s, o);
        cur.finish(a, m * a.K + k, g, rs, s * inv_k);
    }
    if (a.part == nullptr)
        return;
    store_partial(&share[hw][16 * L], acc);
    __syncthreads();
    for (int c = threadIdx.x; c < 256 * G; c += 128) {
        float t = share[c >> 8][c & 255];
#pragma unroll
        for (int i = 1; i < 8 / G; ++i)
            t += share[G * i + (c >> 8)][c & 255];
        a.part[(int64_t)blockIdx.x * a.K + c] = t;
    }
}

// 16384 < K <= 32768: a cluster of five to eight CTAs per row, each with a share
// of its blocks (at most one per half-warp) and of dgamma's partial row; the
// row's sum goes round by shared memory, one cluster barrier a row (the slots
// alternate).  A CTA per row would have to rotate every block twice (16640
// columns, 6049 rows: 463 us against 297).  For 10240 < K <= 16384 two blocks a
// half-warp, some of them spilled, are still faster (12288: 207 us against 258).
template <bool GBF16>
__global__ void __launch_bounds__(256) rmsnorm_backward_cluster_kernel(const BwdArgs a, int ctas)
{
    constexpr int THREADS = 256;
    constexpr int kHalfWarps = THREADS / 16;
    __shared__ __align__(16) float tr_all[kHalfWarps][16 * 16 + 16];
    __shared__ float warp_sum[2][THREADS / 32];
    __shared__ __align__(8) float2 slot_sum[2];  // .x: this CTA's share of the row's sum
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hw = threadIdx.x >> 4, L = threadIdx.x & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1));
    const int rank = (int)cluster_ctarank(), NB = (int)(a.K / 256), per = (NB + ctas - 1) / ctas;
    const int b = rank * per + hw;
    const bool mine = hw < per && b < NB;
    const int64_t k = 256 * (int64_t)b + 16 * L, row0 = blockIdx.x / ctas, step = gridDim.x / ctas;
    const float inv_k = 1.0f / (float)a.K;
    uint64_t acc[8] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
    BwdBlock next;
    float nrs = 0.0f;
    auto fetch = [&](int64_t m) {
        if (m < a.M) {
            nrs = a.rs[m];
            if (mine)
                next.load(a, m * a.K + k);
        }
    };
    fetch(row0);
    int slot = 0;
    for (int64_t m = row0; m < a.M; m += step, slot ^= 1) {
        const BwdBlock cur = next;
        const float rs = nrs;
        fetch(m + step);
        uint64_t g[8], s2 = 0ull;
        if (mine)
            cur.first<GBF16>(a, k, L, tr_all[hw], hmask, pair_both(rs * 0.0625f), g, acc, s2);
        const float own = block_sum<THREADS>(sum_pair(s2), warp_sum, slot);
        if (threadIdx.x == 0)
            slot_sum[slot].x = own;
        __syncwarp();
        cluster_sync();
        // lane r of every warp fetches CTA r's share (one remote load in flight a
        // warp, not one after another), added by a butterfly
        const int lane = threadIdx.x & 31;
        float sum = 0.0f;
        if (lane < ctas)
            sum = ld_cluster_f2(mapa_shared(smem_u32(&slot_sum[slot]), (uint32_t)lane)).x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (mine)
            cur.finish(a, m * a.K + k, g, rs, sum * inv_k);
    }
    if (a.part != nullptr && mine)
        store_partial(a.part + row0 * a.K + k, acc);
    __syncwarp();
    cluster_sync();  // nobody leaves while its shared memory may be read
}

// One CTA per row at a time, J blocks per half-warp (512 < K <= 16384); with one
// block the next row's values are loaded while the current row is worked on.
// J = 1 up to 10240 columns, with as few warps as the row takes (39321 x 2560:
// 170 us with 256 threads, 140 with 160; 9728 columns: 238 us with two blocks a
// half-warp, 182 with one in 640 threads); one block in 704 threads, which leave
// 80 registers, was slower than two (11008: 232 us against 223).
// (Written out, not with BwdBlock: the compiler kept the struct form's registers
// in another order, and 8192 x 4096 took 57 us instead of 51.)
template <int J, int THREADS, bool GBF16>
__global__ void __launch_bounds__(THREADS, THREADS == 320 ? 2 : 0) rmsnorm_backward_kernel(const BwdArgs a)
{
    constexpr int kHalfWarps = THREADS / 16;
    __shared__ __align__(16) float tr_all[kHalfWarps][16 * 16 + 16];
    __shared__ float warp_sum[2][THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int tid = threadIdx.x, hw = tid >> 4, L = tid & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1));
    const int NB = (int)(a.K / 256);
    const float inv_k = 1.0f / (float)a.K;
    float *tr = tr_all[hw];
    float *prow = a.part != nullptr ? a.part + (int64_t)blockIdx.x * a.K : nullptr;
    uint64_t acc[J][8];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[j][i] = 0ull;

    auto rotated = [&](const uint32_t (&w)[8], uint64_t (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = pair_of(w[i]);
        rotate_rows16(L, tr, hmask, v);
    };
    auto finish = [&](int64_t at, const uint64_t (&g)[8], const uint32_t (&hp)[8], const uint32_t (&r)[8], float rs,
                      float c) {
        const uint64_t rs16 = pair_both(rs * 0.0625f), k = pair_both(-16.0f * c * rs);
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo, hi;
            unpack2(fma2(fma2(pair_of(hp[i]), k, g[i]), rs16, pair_of(r[i])), lo, hi);
            o[i] = to_bf16x2_bits(__uint_as_float(lo), __uint_as_float(hi));
        }
        store16(a.dx + at, a.wide, o);
    };
    int slot = 0;
    // the next row's values are loaded while the current row is worked on
    uint32_t nd[J][8], nh[J][8], nr[J][8];
    float nrs = 0.0f;
    auto fetch = [&](int64_t m) {
        if (m >= a.M)
            return;
        nrs = a.rs[m];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int b = hw + kHalfWarps * j;
            if (b < NB) {
                const int64_t at = m * a.K + 256 * b + 16 * L;
                load16(a.dr + at, a.wide, nd[j]);
                load16(a.h + at, a.wide, nh[j]);
                if (a.dres != nullptr) {
                    load16(a.dres + at, a.wide, nr[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        nr[j][i] = 0u;
                }
            }
        }
    };
    constexpr bool kAhead = J == 1;  // two blocks a half-warp leave no registers for it
    if (kAhead)
        fetch(blockIdx.x);
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, slot ^= 1) {
        if (!kAhead)
            fetch(m);
        const float rs = nrs;
        const uint64_t rs16 = pair_both(rs * 0.0625f);
        uint64_t s = 0ull, g[J][8];
        uint32_t hp[J][8], r[J][8], d[J][8];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[j][i] = nd[j][i];
                hp[j][i] = nh[j][i];
                r[j][i] = nr[j][i];
            }
        if (kAhead)
            fetch(m + gridDim.x);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int b = hw + kHalfWarps * j;
            if (b < NB) {
                rotated(d[j], g[j]);
                uint64_t gm[8];
                load_gamma_pairs<GBF16>(a.gamma, 256 * b + 16 * L, gm);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint64_t xh = mul2(pair_of(hp[j][i]), rs16);
                    acc[j][i] = fma2(g[j][i], xh, acc[j][i]);
                    g[j][i] = mul2(g[j][i], gm[i]);
                    s = fma2(g[j][i], xh, s);
                }
            }
        }
        const float c = block_sum<THREADS>(sum_pair(s), warp_sum, slot) * inv_k;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int b = hw + kHalfWarps * j;
            if (b < NB)
                finish(m * a.K + 256 * b + 16 * L, g[j], hp[j], r[j], rs, c);
        }
    }
    if (prow != nullptr) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int b = hw + kHalfWarps * j;
            if (b < NB) {
                ulonglong2 *pp = reinterpret_cast<ulonglong2 *>(prow + 256 * b + 16 * L);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    pp[q] = make_ulonglong2(acc[j][2 * q], acc[j][2 * q + 1]);
            }
        }
    }
}

// Rows longer than a cluster holds (K > 32768): every block is read and rotated
// twice, and the CTA's partial row of dgamma is added to in memory by the
// thread that owns the element (65536 columns, 1536 rows: 365 us; a cluster of
// CTAs of 512 threads took 529).
template <bool GBF16>
__global__ void __launch_bounds__(512) rmsnorm_backward_wide_kernel(const BwdArgs a)
{
    constexpr int kHalfWarps = 32;
    __shared__ __align__(16) float tr_all[kHalfWarps][16 * 16 + 16];
    __shared__ float warp_sum[2][16];
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hw = threadIdx.x >> 4, L = threadIdx.x & 15;
    const unsigned hmask = 0xFFFFu << (16 * (hw & 1));
    const int NB = (int)(a.K / 256);
    const float inv_k = 1.0f / (float)a.K;
    int slot = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, slot ^= 1) {
        const float rs = a.rs[m];
        const uint64_t rs16 = pair_both(rs * 0.0625f);
        uint64_t g[8], s2 = 0ull;
        BwdBlock blk;
        for (int b = hw; b < NB; b += kHalfWarps) {
            const int64_t k = 256 * (int64_t)b + 16 * L;
            float *pp = a.part != nullptr ? a.part + (int64_t)blockIdx.x * a.K + k : nullptr;
            uint64_t acc[8] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
            if (pp != nullptr && m != blockIdx.x) {
                const ulonglong2 *p2 = reinterpret_cast<const ulonglong2 *>(pp);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const ulonglong2 t = p2[q];
                    acc[2 * q] = t.x;
                    acc[2 * q + 1] = t.y;
                }
            }
            blk.load(a, m * a.K + k);
            blk.first<GBF16>(a, k, L, tr_all[hw], hmask, rs16, g, acc, s2);
            if (pp != nullptr)
                store_partial(pp, acc);
        }
        const float c = block_sum<512>(sum_pair(s2), warp_sum, slot) * inv_k;
        for (int b = hw; b < NB; b += kHalfWarps) {
            const int64_t k = 256 * (int64_t)b + 16 * L;
            uint64_t acc[8] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
            blk.load(a, m * a.K + k);
            blk.first<GBF16>(a, k, L, tr_all[hw], hmask, rs16, g, acc, s2);
            blk.finish(a, m * a.K + k, g, rs, c);
        }
    }
}

// dgamma[k] = sum over p of part[p, k], in a fixed order: a CTA takes 32
// columns, its 32 warps every 32nd partial row each, then one warp adds the 32
// (with eight warps the chain of loads took 9 us of the 8192 x 4096 gradient,
// cold).
constexpr int kSumWarps = 32;

__global__ void __launch_bounds__(32 * kSumWarps) dgamma_kernel(const float *__restrict__ part, int P, int64_t K,
                                                                float *__restrict__ dgamma)
{
    __shared__ float sh[kSumWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t k = 32 * (int64_t)blockIdx.x + lane;  // K is a multiple of 256
    float s = 0.0f;
#pragma unroll 8
    for (int p = w; p < P; p += kSumWarps)
        s += part[(int64_t)p * K + k];
    sh[w][lane] = s;
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int i = 1; i < kSumWarps; ++i)
            s += sh[i][lane];
        dgamma[k] = s;
    }
}

// CTAs of a row's cluster for 16384 < K <= 32768: 4096 columns (256 threads, two
// CTAs an SM) each.
inline int cluster_ctas(int64_t K) { return (int)((K + 4095) / 4096); }

// Row groups of the backward's grid (CTAs, or clusters), and with it the
// partial rows of dgamma: a function of the shape alone, so that the caller's
// workspace has a fixed size.  All groups are resident from the start: 16 warps
// an SM at up to 128 registers, 20 at up to 96 (the registers are dealt out by
// quarters of an SM; one CTA of 96 threads too many, and 65536 x 1536 took 184
// us instead of 137).  A cluster's CTAs share a GPC; eight GPCs of at least 16
// SMs are counted on (with two clusters more than fit, 16384 took twice the
// time).
inline int64_t backward_groups(int64_t M, int64_t K)
{
    const int64_t nb = K / 256;
    const int64_t most = nb <= 2    ? 148 * 4
                         : nb <= 4  ? 148 * 8
                         : nb <= 6  ? 148 * 5
                         : nb <= 8  ? 148 * 4
                         : nb <= 12 ? 148 * 3
                         : nb <= 20 ? 148 * 2
                         : nb > 64 && nb <= 128 ? 32 / cluster_ctas(K) * 8
                                                : 148;
    const int64_t rows = K == 256 ? 8 : K == 512 ? 4 : 1;  // a group's rows at once
    const int64_t need = (M + rows - 1) / rows;
    return need < most ? need : most;
}

// A launch in clusters, as a programmatic dependent.
template <class... Args>
inline cudaError_t launch_clusters(void (*kern)(Args...), int64_t clusters, int ctas, int threads, cudaStream_t stream,
                                   Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * ctas));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool GBF16>
inline cudaError_t launch_bwd_t(const BwdArgs &a, float *dgamma, cudaStream_t stream)
{
    const int64_t P = backward_groups(a.M, a.K);
    const dim3 grid((unsigned)P);
    auto in_one = [&](auto threads) {  // a half-warp per block
        constexpr int T = decltype(threads)::value;
        return launch_dependent(rmsnorm_backward_kernel<1, T, GBF16>, grid, T, 0, stream, a);
    };
    cudaError_t e;
    const int64_t nb = a.K / 256;
    if (nb == 1)
        e = launch_dependent(rmsnorm_backward_small_kernel<1, GBF16>, grid, 128, 0, stream, a);
    else if (nb == 2)
        e = launch_dependent(rmsnorm_backward_small_kernel<2, GBF16>, grid, 128, 0, stream, a);
    else if (nb <= 4)
        e = in_one(std::integral_constant<int, 64>{});
    else if (nb <= 6)
        e = in_one(std::integral_constant<int, 96>{});
    else if (nb <= 8)
        e = in_one(std::integral_constant<int, 128>{});
    else if (nb <= 10)
        e = in_one(std::integral_constant<int, 160>{});
    else if (nb <= 12)
        e = in_one(std::integral_constant<int, 192>{});
    else if (nb <= 16)
        e = in_one(std::integral_constant<int, 256>{});
    else if (nb <= 20)
        e = in_one(std::integral_constant<int, 320>{});
    else if (nb <= 32)
        e = in_one(std::integral_constant<int, 512>{});
    else if (nb <= 40)
        e = in_one(std::integral_constant<int, 640>{});
    else if (nb <= 64)
        e = launch_dependent(rmsnorm_backward_kernel<2, 512, GBF16>, grid, 512, 0, stream, a);
    else if (nb <= 128)
        e = launch_clusters(rmsnorm_backward_cluster_kernel<GBF16>, P, cluster_ctas(a.K), 256, stream, a,
                            cluster_ctas(a.K));
    else
        e = launch_dependent(rmsnorm_backward_wide_kernel<GBF16>, grid, 512, 0, stream, a);
    if (e != cudaSuccess || dgamma == nullptr)
        return e;
    return launch_dependent(dgamma_kernel, dim3((unsigned)(a.K / 32)), 32 * kSumWarps, 0, stream, (const float *)a.part,
                            (int)P, a.K, dgamma);
}

inline cudaError_t launch_bwd(BwdArgs a, bool gamma_bf16, float *dgamma, cudaStream_t stream)
{
    a.wide = all_wide({a.dr, a.h, a.dres, a.dx});
    return gamma_bf16 ? launch_bwd_t<true>(a, dgamma, stream) : launch_bwd_t<false>(a, dgamma, stream);
}

}  // namespace nm
}  // namespace cr

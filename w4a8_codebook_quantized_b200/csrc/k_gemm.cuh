// k_gemm.cuh -- prefill contraction on the 5th-generation tensor cores.
//
// What it computes (ai-toolkit convrot_w4a8_quant.py, _w4a8_linear_ste_op:
// torch._int_mm(aq, w8.t()) followed by the epilogue):
//   acc[m, n] = sum_k A[m, k] * B[n, k]   A = xq [M, K] int8, B = w8 [N, K] int8
//   out[m, n] = float(acc) * (xs[m] * ws[n]) [+ bias[n]]
//
// and, on the same pipeline, what the gradients and the loss around that layer
// contract (Mode below): the gated layer's gradient and the cross entropy's
// statistics and gradient as epilogues of the int8 contraction, and their bf16
// input-gradient contractions.
//
// B200 design: a persistent, warp-specialised kernel, one CTA per SM.
//   warp 0      one thread issues TMA loads of 128-wide K slices of the A tile
//               (128 rows) and the B tile (256 rows) into a 4-stage ring of
//               128-byte-swizzled shared-memory buffers (48 KB per stage);
//   warp 1      allocates 512 TMEM columns (two 128 x 256 int32 accumulators)
//               and one thread issues tcgen05.mma kind::i8 (M 128, N 256, K 32,
//               four per stage), releasing each stage with tcgen05.commit;
//   warps 2-5   (2-9, epi_warps) the epilogue: tcgen05.ld of 32 columns at a
//               time, the per-token x per-channel fp32 rescale (+ bias), bf16 or
//               fp32 stores, then the TMEM buffer is handed back to the MMA
//               warp, so the epilogue of tile i overlaps the MMAs of tile i + 1.
// What bounds it: four MMAs of a stage take some 512 cycles of the tensor core,
// and the issuing thread's own instructions come near that when the epilogue's
// warps compete for its scheduler.  Ready descriptors in uniform registers, one
// commit for both CTAs, and packed arithmetic in the epilogues took the gated
// gradient's int8 part (4096 x 12288 x 4096) from 167 to 136 us, the tensor pipe
// from 62 to 80 percent busy; the rest is the clock, 1.5 to 1.6 GHz under the
// power limit.
// Every wait is bounded (a second or two); a wait that runs out sets the
// library error word, every role stops, TMEM is freed and the kernel returns.
// TMA zero-fills rows past M or N, so ragged edges need no special casing
// except in the epilogue's stores.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cr_device.cuh"

namespace cr {
namespace gm {

// What a GEMM's operands are and what its epilogue does with the accumulators.
enum Mode : int {
    kI8 = 0,         // int8; the layer's outputs (with SwiGLU when asked)
    kBf16 = 1,       // bf16 x bf16 -> fp32; the accumulators are the outputs
    kBf16RowsAdd = 2,  // bf16; outputs scaled by row and added to the fp32 outputs already there
    kSwigluGrad = 3, // int8; the gradient of interleaved gate/up outputs
    kCeStats = 4,    // int8; softmax statistics of the outputs
    kCeGrad = 5,     // int8; the cross entropy's gradient of the outputs, up to each row's factor
    kBf16Rows = 6,   // bf16; outputs scaled by row
    kBf16Nt = 7,     // bf16; as kBf16, with B as below
    kModes = 8
};

constexpr bool is_bf16(int mode)
{
    return mode == kBf16 || mode == kBf16Nt || mode == kBf16Rows || mode == kBf16RowsAdd;
}
// B is given as [K, N] (N contiguous: an MN-major operand), not as [N, K]: a
// weight [outputs, inputs] is the B of its input gradient as it stands.
constexpr bool b_is_kn(int mode) { return mode == kBf16Nt || mode == kBf16Rows || mode == kBf16RowsAdd; }
constexpr bool row_factor(int mode) { return mode == kBf16Rows || mode == kBf16RowsAdd; }

// The modes whose kernels follow one another in one call (decode -> int8
// contraction -> bf16 contraction -> sum) are launched as programmatic
// dependents: a kernel's launch and set-up overlap its predecessor's tail, and
// it waits for the predecessor before it reads or writes anything.
constexpr bool dependent(int mode) { return mode != kI8 && mode != kBf16; }

// Eight warps for the epilogues that evaluate exponentials per output (each 32
// rows x half a tile's columns) and those of split contractions, where the
// layer's own takes four (32 rows x all columns): with four, the epilogue of an
// int8 tile outlasted the tile's own MMAs, and a split tile's took as long as
// its range of the reduction.
constexpr bool has_exponentials(int mode) { return mode == kSwigluGrad || mode == kCeStats || mode == kCeGrad; }
constexpr int epi_warps(int mode) { return mode == kI8 || mode == kBf16 ? 4 : 8; }
constexpr int threads(int mode) { return 64 + 32 * epi_warps(mode); }

// Where a tile's column j has its scale and bias in shared memory: for the
// gated gradient in the order gate, gate, up, up of two pairs of columns.
template <int MODE>
__device__ __forceinline__ int stage_column(int j)
{
    return MODE == kSwigluGrad && ((j & 3) == 1 || (j & 3) == 2) ? j ^ 3 : j;
}

// What the epilogues beyond the layer's own read and write.
struct EpiArgs {
    const uint16_t *dout = nullptr;    // kSwigluGrad: [M, N / 2] bf16
    const int64_t *targets = nullptr;  // kCe*: [M]
    int64_t ignore = 0, V = 0;         // kCe*: the target that has no loss; the whole vocabulary
    int n0 = 0;                        // kCe*: the vocabulary entry of column 0
    float2 *part = nullptr;            // kCeStats: [M, slices] (reference in log2, sum)
    int slices = 0;
    float *tlogit = nullptr;           // kCeStats: [M], the target's output
    const float *lse = nullptr;        // kCeGrad: [M]
    const float *dloss = nullptr;      // kBf16Rows*: [M], with targets
    // modes with B as [K, N]: how tiles are spread over the SMs (Tiling)
    int slots = 1, max_splits = 1, split_tail = 0;
    const int *count = nullptr;        // the number of rows where it is known on the device only

    // Whether a row of the cross entropy's gradient takes part in the loss, and
    // its factor then: dloss, NaN where the target is outside the vocabulary.
    __device__ __forceinline__ bool takes_part(int row, float &factor) const
    {
        const int64_t t = targets[row];
        if (t == ignore)
            return false;
        factor = t >= 0 && t < V ? dloss[row] : __int_as_float(0x7FC00000);
        return true;
    }
};

constexpr int kSlotCols = 256;  // = BN

// The order of tiles: kGroup tile rows at a time, column by column, so that
// the tiles in flight (one wave) form a block of about kGroup x 9 tiles and
// every operand line is wanted by several SMs at about the same time.  Measured
// against row by row (1): 4096 x 65536 x 4096 cross-entropy gradient 2735 ->
// 2675 us, the others within 1 percent; 4 and 16 were slower on the gated layer.
constexpr int kGroup = 8;

__host__ __device__ __forceinline__ void tile_place(int tile, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int per_group = kGroup * tiles_n, g = tile / per_group, r = tile - g * per_group;
    const int rows = tiles_m - g * kGroup < kGroup ? tiles_m - g * kGroup : kGroup;
    tn = r / rows;
    tm = g * kGroup + r - tn * rows;
}

__host__ __device__ __forceinline__ int tile_number(int tm, int tn, int tiles_m, int tiles_n)
{
    const int g = tm / kGroup, rows = tiles_m - g * kGroup < kGroup ? tiles_m - g * kGroup : kGroup;
    return g * kGroup * tiles_n + tn * rows + tm - g * kGroup;
}

// The units of work of a contraction with B as [K, N].  A unit is a tile, or
// one of `splits` ranges of the reduction of a tile of the last, partial wave
// (all tiles, where they do not fill one wave of `slots` SMs or SM pairs): those
// ranges run beside one another, each into an fp32 copy of the tile of its own,
// and split_sum_kernel adds them up in order.  A range of a short last piece of
// the reduction may be empty.
struct Tiling {
    int tiles_m, tiles_n, kblocks, full, splits, units;

    __host__ __device__ Tiling(int M, int N, int kb, int bm, int slots, int max_splits, int split_tail,
                               int cols = kSlotCols)
    {
        tiles_n = (N + cols - 1) / cols;
        kblocks = kb;
        tiles_m = (M + bm - 1) / bm;
        const int tiles = tiles_m * tiles_n;
        const int tail = tiles < slots || split_tail ? tiles % slots : 0;
        splits = tail ? slots / tail : 1;
        if (splits > max_splits)
            splits = max_splits;
        full = splits > 1 ? tiles - tail : tiles;
        units = full + (tiles - full) * splits;
    }

    // A unit's tile and its range [k0, k1) of the reduction's blocks; `copy` is
    // its fp32 copy's number, -1 for a whole tile.  False: an empty range.
    __device__ __forceinline__ bool at(int unit, int &tm, int &tn, int &k0, int &k1, int &copy) const
    {
        int tile = unit;
        k0 = 0;
        k1 = kblocks;
        copy = -1;
        if (unit >= full) {
            copy = unit - full;
            const int t = copy / splits, s = copy - t * splits;
            tile = full + t;
            k0 = (int)((int64_t)kblocks * s / splits);
            k1 = (int)((int64_t)kblocks * (s + 1) / splits);
        }
        tile_place(tile, tiles_m, tiles_n, tm, tn);
        return k0 < k1;
    }
};

constexpr int BM = 128, BN = 256, BK = 128;  // BK in int8 elements = bytes
constexpr int kABytes = BM * BK;              // 16 KB
constexpr int kKnBytes = 64 * 128;            // 8 KB: 64 terms x 64 columns of a B given as [K, N]
constexpr int kEpiBytes = 32 * 128;           // one epilogue store unit: 32 rows x 128 bytes

// Staging of the epilogue: a 4 KB unit per warp, half of one where the warps
// of the epilogues with exponentials store 64 bytes a row.
constexpr int epi_units(int mode) { return has_exponentials(mode) ? epi_warps(mode) / 2 : epi_warps(mode); }
// Per-tile channel scales: none in the modes that have no use for them.
constexpr int scale_cols(int mode, int tn) { return b_is_kn(mode) ? 4 : tn; }

// One CTA's shared memory for 128 x TN tiles (TN 256, or 128 for problems of
// few tiles): a ring of 4 or 6 stages, 192 KB.
template <int MODE, int TN>
struct __align__(1024) Smem {
    static constexpr int kStages = TN == 256 ? 4 : 6;
    static constexpr int kStageBytes = kABytes + TN * BK;
    static constexpr int kTmemCols = 2 * TN;  // two accumulators
    uint8_t stage[kStages][kStageBytes];           // A at +0, B at +kABytes; every buffer 1024-aligned
    uint8_t epi[epi_units(MODE)][kEpiBytes];       // swizzled staging units
    float wsb[2][scale_cols(MODE, TN)];            // per-tile channel scales (double-buffered by tile parity)
    float biasb[2][scale_cols(MODE, TN)];          // per-tile bias
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint32_t tmem_base;
    int abort;
};

constexpr size_t kMaxSmem = 227 * 1024;  // per CTA

template <int MODE, int TN>
constexpr size_t smem_bytes()
{
    static_assert(sizeof(Smem<MODE, TN>) + 1024 <= kMaxSmem, "shared memory of one CTA");
    return sizeof(Smem<MODE, TN>) + 1024;  // + slack to align the base
}

static_assert(BN == kSlotCols, "tile width of Tiling");

// Rows of the boxes that bring A to a 128-row tile: 128, or where A has fewer
// rows no more than those (the tile's other rows hold whatever was there; they
// belong to no row of the output).  Rows that a box fills past the tensor's end
// are not free: with boxes of 128 rows 9 x 32768 x 4096 takes 36.9 us instead of
// 29.5, 32 rows the same.
__host__ __device__ constexpr int a_box_rows(int64_t M) { return M < BM ? (int)(M + 7) / 8 * 8 : BM; }

__device__ __forceinline__ void tile_coords(int tile, int tiles_n, int &tm, int &tn)
{
    tm = tile / tiles_n;
    tn = tile - tm * tiles_n;
}

// One 128-byte unit (32 words a lane) of a warp's 32 rows -> staging buffer ->
// TMA bulk store (ADD: bulk reduction, fp32 addition in memory).
template <bool ADD>
__device__ __forceinline__ void store_unit_rows(const uint32_t (&p)[32], int ucol0, int row0, int lane,
                                                const CUtensorMap *tmOut, uint8_t *stg, uint32_t &units_issued)
{
    if (units_issued >= 1) {
        if (lane == 0)
            bulk_wait_read<0>();  // the previous store has read the staging buffer
        __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(stg + lane * 128 + ((c ^ (lane & 7)) * 16)) =
            make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        if constexpr (ADD)
            tma_add_2d(tmOut, ucol0, row0, stg);
        else
            tma_store_2d(tmOut, ucol0, row0, stg);
        bulk_commit();
    }
    ++units_issued;
}

// The same for 32 bf16 columns (16 words a lane, 64 bytes a row; `tmOut` has
// the 64-byte swizzle: chunk c of row r at chunk c ^ ((r / 2) % 4)).
__device__ __forceinline__ void store_half_unit(const uint32_t (&p)[16], int ucol0, int row0, int lane,
                                                const CUtensorMap *tmOut, uint8_t *stg, uint32_t &units_issued)
{
    if (units_issued >= 1) {
        if (lane == 0)
            bulk_wait_read<0>();  // the previous store has read the staging buffer
        __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4 *>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16)) =
            make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(tmOut, ucol0, row0, stg);
        bulk_commit();
    }
    ++units_issued;
}

// Epilogue of one 128 x 256 accumulator tile for one warp: its 32 TMEM lanes
// are rows row0 + lane; `tbase` addresses lane 0 of the warp's quarter at the
// tile's first column; the output columns are col_base + [0, 256).  Fast path
// (tma_out): 128-byte column units (64 bf16 or 32 fp32 columns) go through the
// 128B-swizzled staging buffer `stage_buf` (16-byte chunk c of row r at chunk
// c ^ (r % 8): conflict-free) and one TMA bulk store each; the next 32-column
// TMEM load is in flight while the current chunk is converted.  Otherwise each
// thread stores its own row.  release() hands the accumulator back once every
// column is in registers.
// RAW: the accumulator holds fp32 values that are the outputs themselves
// (bf16 GEMM; ROWS: times xm, and 0 in rows without row_ok, whose values may be
// NaN); no channel scales, bias or SwiGLU.  ADD: the fp32 outputs are added to
// what is there, by the bulk stores' own reduction (tma_out only).
template <bool RAW, bool ROWS, bool ADD, int COLS, class Release>
__device__ __forceinline__ void epilogue_tile(uint32_t tbase, int row0, int col_base, int lane, float xm, bool row_ok,
                                              const float *wsv, const float *bsv, bool has_bias, int M, int N,
                                              int out_f32, int swiglu, int tma_out, const CUtensorMap *tmOut,
                                              uint8_t *stage_buf,
                                              uint32_t &units_issued, void *__restrict__ out,
                                              int32_t *__restrict__ acc_out, const float *__restrict__ ws,
                                              const float *__restrict__ bias, Release release)
{
    const int row = row0 + lane;
    // 32 accumulators of columns [c0, c0 + 32) of the tile -> 32 fp32 or 16 bf16x2 words
    auto convert32 = [&](const uint32_t (&v)[32], int c0, uint32_t *dst) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            float y[4];
            if constexpr (RAW) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = !ROWS    ? __uint_as_float(v[j + e])
                           : row_ok ? __fmul_rn(__uint_as_float(v[j + e]), xm)
                                    : 0.0f;
            } else {
                const float4 w4 = *reinterpret_cast<const float4 *>(wsv + c0 + j);
                const float4 b4 = *reinterpret_cast<const float4 *>(bsv + c0 + j);
                const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
                const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = __fmul_rn(__int2float_rn((int32_t)v[j + e]), __fmul_rn(xm, wv[e]));
                    if (has_bias)
                        y[e] = __fadd_rn(y[e], bv[e]);
                }
            }
            if (out_f32) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dst[j + e] = __float_as_uint(y[e]);
            } else {
                dst[j / 2] = to_bf16x2_bits(y[0], y[1]);
                dst[j / 2 + 1] = to_bf16x2_bits(y[2], y[3]);
            }
        }
    };
    auto store_unit = [&](const uint32_t (&p)[32], int ucol0) {
        store_unit_rows<ADD>(p, ucol0, row0, lane, tmOut, stage_buf, units_issued);
    };
    uint32_t cur[32], nxt[32], packed[32];
    if (!RAW && swiglu) {
        // Interleaved gate/up rows: accumulator columns 2f and 2f + 1 are one
        // pair and give output column f of [M, N / 2].  Each 32-column TMEM
        // load yields 16 outputs; a 128-byte unit (64 bf16 or 32 fp32 outputs)
        // takes 4 or 2 loads.
        const int F = N >> 1, ocol_base = col_base >> 1;
        auto pairs16 = [&](int c0, float (&y)[16]) {
#pragma unroll
            for (int p = 0; p < 16; ++p) {
                float g = __fmul_rn(__int2float_rn((int32_t)cur[2 * p]), __fmul_rn(xm, wsv[c0 + 2 * p]));
                float u = __fmul_rn(__int2float_rn((int32_t)cur[2 * p + 1]), __fmul_rn(xm, wsv[c0 + 2 * p + 1]));
                if (has_bias) {
                    g = __fadd_rn(g, bsv[c0 + 2 * p]);
                    u = __fadd_rn(u, bsv[c0 + 2 * p + 1]);
                }
                y[p] = swiglu_value(g, u);
            }
        };
        // uo: output columns per 128-byte unit (compile-time, so that `packed`
        // stays in registers)
        auto units = [&](auto uo_c) {
            constexpr int uo = decltype(uo_c)::value;
            for (int un = 0; un < COLS / (2 * uo); ++un) {
#pragma unroll
                for (int k = 0; k < uo / 16; ++k) {
                    const int c0 = 2 * uo * un + 32 * k;
                    __syncwarp();
                    tmem_ld_32cols(tbase + (uint32_t)c0, cur);
                    tmem_ld_wait();
                    if (c0 + 32 == COLS)
                        release();
                    float y[16];
                    pairs16(c0, y);
                    if constexpr (uo == 32) {
#pragma unroll
                        for (int p = 0; p < 16; ++p)
                            packed[16 * k + p] = __float_as_uint(y[p]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            packed[8 * k + i] = to_bf16x2_bits(y[2 * i], y[2 * i + 1]);
                    }
                }
                store_unit(packed, ocol_base + uo * un);
            }
        };
        if (tma_out && out_f32) {
            units(std::integral_constant<int, 32>{});
        } else if (tma_out) {
            units(std::integral_constant<int, 64>{});
        } else {
            for (int ch = 0; ch < COLS / 32; ++ch) {
                const int c0 = 32 * ch;
                __syncwarp();
                tmem_ld_32cols(tbase + (uint32_t)c0, cur);
                tmem_ld_wait();
                if (ch + 1 == COLS / 32)
                    release();
                float y[16];
                pairs16(c0, y);
                const int f0 = ocol_base + 16 * ch;
                if (row_ok && f0 < F) {
                    const int64_t base = (int64_t)row * F + f0;
#pragma unroll
                    for (int p = 0; p < 16; ++p) {
                        if (f0 + p >= F)
                            break;
                        if (out_f32)
                            reinterpret_cast<float *>(out)[base + p] = y[p];
                        else
                            reinterpret_cast<uint16_t *>(out)[base + p] = to_bf16_bits(y[p]);
                    }
                }
            }
        }
        return;
    }
    __syncwarp();
    tmem_ld_32cols(tbase, cur);
    tmem_ld_wait();
    if (tma_out && !out_f32) {
        // units of 64 columns: two 32-column chunks each
        for (int u = 0; u < COLS / 64; ++u) {
            __syncwarp();
            tmem_ld_32cols(tbase + (uint32_t)(64 * u + 32), nxt);
            convert32(cur, 64 * u, packed);
            tmem_ld_wait();
            if (u + 1 < COLS / 64) {
                __syncwarp();
                tmem_ld_32cols(tbase + (uint32_t)(64 * u + 64), cur);
            } else {
                release();
            }
            convert32(nxt, 64 * u + 32, packed + 16);
            store_unit(packed, col_base + 64 * u);
            if (u + 1 < COLS / 64)
                tmem_ld_wait();
        }
    } else if (tma_out) {
        // units of 32 fp32 columns
        for (int u = 0; u < COLS / 32; ++u) {
            if (u + 1 < COLS / 32) {
                __syncwarp();
                tmem_ld_32cols(tbase + (uint32_t)(32 * u + 32), nxt);
            } else {
                release();
            }
            convert32(cur, 32 * u, packed);
            store_unit(packed, col_base + 32 * u);
            if (u + 1 < COLS / 32) {
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    cur[j] = nxt[j];
            }
        }
    } else {
        for (int ch = 0; ch < COLS / 32; ++ch) {
            if (ch + 1 < COLS / 32) {
                __syncwarp();
                tmem_ld_32cols(tbase + (uint32_t)(32 * (ch + 1)), nxt);
            } else {
                release();
            }
            const int col0 = col_base + 32 * ch;
            if (row_ok && col0 < N) {
                const int64_t base = (int64_t)row * N + col0;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int n = col0 + j;
                    if (n >= N)
                        break;
                    const float y = ROWS  ? __fmul_rn(__uint_as_float(cur[j]), xm)
                                    : RAW ? __uint_as_float(cur[j])
                                          : epilogue_value((int32_t)cur[j], xm, ws[n], bias, n);
                    if (out_f32)
                        reinterpret_cast<float *>(out)[base + j] = y;
                    else
                        reinterpret_cast<uint16_t *>(out)[base + j] = to_bf16_bits(y);
                    if (acc_out != nullptr)
                        acc_out[base + j] = (int32_t)cur[j];
                }
            }
            if (ch + 1 < COLS / 32) {
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    cur[j] = nxt[j];
            }
        }
    }
}

// The epilogues beyond the layer's own work on pairs of values in packed fp32x2
// arithmetic (each half rounded as the scalar instruction rounds it): their
// warps share the schedulers with the thread that issues the MMAs, and what
// they do not issue, it can.

// Two fp32 outputs of a row as the layer's epilogue computes them, from their
// accumulators and the channels' scales (and bias).
__device__ __forceinline__ uint64_t output_pair(uint32_t a, uint32_t b, uint64_t xm2, uint64_t w2, uint64_t b2,
                                                bool has_bias)
{
    const uint64_t acc = pack2(__float_as_uint(__int2float_rn((int32_t)a)), __float_as_uint(__int2float_rn((int32_t)b)));
    const uint64_t y = mul2(acc, mul2(xm2, w2));
    return has_bias ? add2(y, b2) : y;
}

// The 32 outputs of accumulator columns [c0, c0 + 32) of one row, neighbours
// paired (wsv, bsv: the tile's channel scales and bias).
__device__ __forceinline__ void outputs32(const uint32_t (&v)[32], int c0, uint64_t xm2, const float *wsv,
                                          const float *bsv, bool has_bias, uint64_t (&y)[16])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(wsv + c0 + 4 * j);
        ulonglong2 b = make_ulonglong2(0ull, 0ull);
        if (has_bias)
            b = *reinterpret_cast<const ulonglong2 *>(bsv + c0 + 4 * j);
        y[2 * j] = output_pair(v[4 * j], v[4 * j + 1], xm2, w.x, b.x, has_bias);
        y[2 * j + 1] = output_pair(v[4 * j + 2], v[4 * j + 3], xm2, w.y, b.y, has_bias);
    }
}

__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

constexpr float kLog2e = 1.4426950408889634f;

// 2^x by the special-function unit (2 ulp; 0 for x = -inf, inf for +inf).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x by the special-function unit (1 ulp; 0 for x = +inf).
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Gradients of silu(g) * u for the gradients d of two such products: with
// s = sigmoid(g), du = d g s and dg = d u s (1 + g (1 - s)), returned as (dg, du)
// in bf16 for each.  s = 1 / (1 + 2^(-g log2 e)) is 0 where the power
// overflows (g below -88).  1 - s is taken as a difference: its error, 2^-24,
// is relative to the 1 that g (1 - s) is added to.
__device__ __forceinline__ void swiglu_grad2(uint64_t g, uint64_t u, uint64_t d, uint32_t &z0, uint32_t &z1)
{
    const uint64_t one = pair_both(1.0f);
    const uint64_t x = mul2(g, pair_both(-kLog2e));
    const uint64_t den = add2(one, pack2(__float_as_uint(ex2(lo_of(x))), __float_as_uint(ex2(hi_of(x)))));
    const uint64_t s = pack2(__float_as_uint(rcp(lo_of(den))), __float_as_uint(rcp(hi_of(den))));
    const uint64_t ds = mul2(d, s);
    const uint64_t dg = mul2(mul2(ds, u), fma2(g, sub2(one, s), one));
    const uint64_t du = mul2(ds, g);
    z0 = to_bf16x2_bits(lo_of(dg), lo_of(du));
    z1 = to_bf16x2_bits(hi_of(dg), hi_of(du));
}

// Sixteen bf16 of a row of dout as eight words, columns [f0, f0 + 16) of
// [M, F]: F % 4 == 0, so 8-byte loads are aligned and a group of four columns
// lies inside the row or past it.
__device__ __forceinline__ void load_dout16(const uint16_t *drow, int f0, int F, bool row_ok, uint32_t (&d)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint2 w = make_uint2(0u, 0u);
        if (row_ok && f0 + 4 * i < F)
            w = __ldg(reinterpret_cast<const uint2 *>(drow + f0 + 4 * i));
        d[2 * i] = w.x;
        d[2 * i + 1] = w.y;
    }
}

// The epilogues below take one warp's 32 rows and columns [c_lo, c_lo + COLS)
// of a tile (half of its columns), 32 at a time.

// Epilogue of kSwigluGrad: accumulator columns 2f and 2f + 1 are gate and up
// of output column f; their gradients leave as the same two columns of dz
// [M, N] bf16.  Each row's 16 values of dout for the next 32 columns are loaded
// while the current ones are used (`dn`: those of the first, loaded by the
// caller before it waits for the accumulator).
template <int COLS, class Release>
__device__ __forceinline__ void epilogue_swiglu_grad(uint32_t tbase, int row0, int col_base, int c_lo, int lane,
                                                     float xm, bool row_ok, const float *wsv, const float *bsv,
                                                     bool has_bias, int N, const EpiArgs &ex, const CUtensorMap *tmOut,
                                                     uint8_t *stage_buf, uint32_t &units_issued, uint32_t (&dn)[8],
                                                     Release release)
{
    const int F = N >> 1;
    const uint64_t xm2 = pair_both(xm);
    const uint16_t *drow = ex.dout + (int64_t)(row0 + lane) * F;
#pragma unroll 1
    for (int c0 = c_lo; c0 < c_lo + COLS; c0 += 32) {
        uint32_t cur[32], d[8], packed[16];
        __syncwarp();
        tmem_ld_32cols(tbase + (uint32_t)c0, cur);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] = dn[i];
        if (c0 + 32 < c_lo + COLS)
            load_dout16(drow, (col_base + c0 + 32) >> 1, F, row_ok, dn);
        tmem_ld_wait();
        if (c0 + 32 == c_lo + COLS)
            release();
        // the tile's scales are staged with the middle two of four columns
        // exchanged (stage_column), so that gates and ups pair with their like
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(wsv + c0 + 4 * p);
            ulonglong2 b = make_ulonglong2(0ull, 0ull);
            if (has_bias)
                b = *reinterpret_cast<const ulonglong2 *>(bsv + c0 + 4 * p);
            const uint64_t g = output_pair(cur[4 * p], cur[4 * p + 2], xm2, w.x, b.x, has_bias);
            const uint64_t u = output_pair(cur[4 * p + 1], cur[4 * p + 3], xm2, w.y, b.y, has_bias);
            swiglu_grad2(g, u, pack2(d[p] << 16, d[p] & 0xFFFF0000u), packed[2 * p], packed[2 * p + 1]);
        }
        if (col_base + c0 < N)
            store_half_unit(packed, col_base + c0, row0, lane, tmOut, stage_buf, units_issued);
    }
}

// A row's sum of exponentials as a pair: the reference (its maximum in the
// base-2 domain) and the sum relative to it.  Joining two rescales the smaller
// reference's sum.
__device__ __forceinline__ void join(float2 &a, const float2 b)
{
    const float m = fmaxf(a.x, b.x);
    const float base = m == __int_as_float(0xFF800000) ? 0.0f : m;
    a.y = a.y * ex2(a.x - base) + b.y * ex2(b.x - base);
    a.x = m;
}

// Epilogue of kCeStats: each row's sum of exponentials over the warp's
// columns, relative to its maximum there.  The reference is kept in the base-2
// domain as the rounded product max * log2(e), and every term is 2^(fma(y,
// log2 e, -reference)), so the pair (reference, sum) carries no error of the
// reference's rounding.  Columns past N are left out; -inf outputs (a bias
// that masks a vocabulary entry) contribute 0, also where there is nothing
// else.  The target's output goes to tlogit.
template <int COLS, class Release>
__device__ __forceinline__ float2 epilogue_ce_stats(uint32_t tbase, int row, int col_base, int c_lo, float xm,
                                                    bool row_ok, const float *wsv, const float *bsv, bool has_bias,
                                                    int N, const EpiArgs &ex, Release release)
{
    const float kNegInf = __int_as_float(0xFF800000);
    const int64_t t = row_ok ? ex.targets[row] : -1, lo = (int64_t)ex.n0 + col_base + c_lo;
    const int tcol = (t >= lo && t < lo + COLS && t - ex.n0 < N) ? c_lo + (int)(t - lo) : -1;
    const uint64_t xm2 = pair_both(xm);
    float ref = kNegInf, tl = 0.0f;
    uint64_t s = 0ull;
#pragma unroll 1
    for (int c0 = c_lo; c0 < c_lo + COLS; c0 += 32) {
        uint32_t cur[32];
        __syncwarp();
        tmem_ld_32cols(tbase + (uint32_t)c0, cur);
        tmem_ld_wait();
        if (c0 + 32 == c_lo + COLS)
            release();
        uint64_t y[16];
        outputs32(cur, c0, xm2, wsv, bsv, has_bias, y);
        if (col_base + c0 + 32 > N) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                y[j] = pack2(col_base + c0 + 2 * j < N ? (uint32_t)y[j] : __float_as_uint(kNegInf),
                          col_base + c0 + 2 * j + 1 < N ? (uint32_t)(y[j] >> 32) : __float_as_uint(kNegInf));
        }
        if (tcol >= c0 && tcol < c0 + 32) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (tcol == c0 + 2 * j)
                    tl = lo_of(y[j]);
                if (tcol == c0 + 2 * j + 1)
                    tl = hi_of(y[j]);
            }
        }
        float m0 = lo_of(y[0]), m1 = hi_of(y[0]);
#pragma unroll
        for (int j = 1; j < 16; ++j) {
            m0 = fmaxf(m0, lo_of(y[j]));
            m1 = fmaxf(m1, hi_of(y[j]));
        }
        const float next = fmaxf(ref, __fmul_rn(fmaxf(m0, m1), kLog2e));
        const float base = next == kNegInf ? 0.0f : next;
        s = mul2(s, pair_both(ex2(ref - base)));  // times 0 at the first chunk
        const uint64_t l2 = pair_both(kLog2e), nb = pair_both(-base);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint64_t x = fma2(y[j], l2, nb);
            s = add2(s, pack2(__float_as_uint(ex2(lo_of(x))), __float_as_uint(ex2(hi_of(x)))));
        }
        ref = next;
    }
    if (tcol >= 0)
        ex.tlogit[row] = tl;
    return make_float2(ref, lo_of(s) + hi_of(s));
}

// Epilogue of kCeGrad: dl[m, n] = e^(y - lse[m]) - [n = target] to bf16 (an
// ignored row's values go nowhere: its outputs are not taken from the sum); columns from N to the buffer's width (a multiple of
// 8) are written as zeros.  The row's factor dloss[m] is applied after the
// contraction: dl at the target is then -1 rounded by at most the target's
// probability, where -dloss itself would carry bf16's relative rounding, the
// same one in every row of a mean (0.4 percent of dx at worst).
template <int COLS, class Release>
__device__ __forceinline__ void epilogue_ce_grad(uint32_t tbase, int row0, int col_base, int c_lo, int lane, float xm,
                                                 bool row_ok, const float *wsv, const float *bsv, bool has_bias,
                                                 int N, const EpiArgs &ex, const CUtensorMap *tmOut,
                                                 uint8_t *stage_buf, uint32_t &units_issued, Release release)
{
    const int row = row0 + lane;
    float lse2 = __int_as_float(0x7F800000);  // an ignored row: every exponential 0, where its outputs are finite
    int tcol = -1;
    if (row_ok) {
        const int64_t t = ex.targets[row];
        if (t != ex.ignore) {
            lse2 = __fmul_rn(ex.lse[row], kLog2e);
            const int64_t lo = (int64_t)ex.n0 + col_base;
            tcol = (t >= lo && t < lo + 2 * COLS) ? (int)(t - lo) : -1;
        }
    }
    const uint64_t xm2 = pair_both(xm), nlse = pair_both(-lse2);
#pragma unroll 1
    for (int c0 = c_lo; c0 < c_lo + COLS; c0 += 32) {
        uint32_t cur[32], packed[16];
        __syncwarp();
        tmem_ld_32cols(tbase + (uint32_t)c0, cur);
        tmem_ld_wait();
        if (c0 + 32 == c_lo + COLS)
            release();
        uint64_t y[16];
        outputs32(cur, c0, xm2, wsv, bsv, has_bias, y);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint64_t x = fma2(y[j], pair_both(kLog2e), nlse);
            y[j] = pack2(__float_as_uint(ex2(lo_of(x))), __float_as_uint(ex2(hi_of(x))));
        }
        if (tcol >= c0 && tcol < c0 + 32) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                y[j] = add2(y[j], pack2(tcol == c0 + 2 * j ? __float_as_uint(-1.0f) : 0u,
                                        tcol == c0 + 2 * j + 1 ? __float_as_uint(-1.0f) : 0u));
        }
        if (col_base + c0 + 32 > N) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                y[j] = pack2(col_base + c0 + 2 * j < N ? (uint32_t)y[j] : 0u,
                          col_base + c0 + 2 * j + 1 < N ? (uint32_t)(y[j] >> 32) : 0u);
        }
#pragma unroll
        for (int p = 0; p < 16; ++p)
            packed[p] = to_bf16x2_bits(lo_of(y[p]), hi_of(y[p]));
        if (col_base + c0 < N)
            store_half_unit(packed, col_base + c0, row0, lane, tmOut, stage_buf, units_issued);
    }
}

// One tile's epilogue for one warp of the CTA's epilogue warps, by mode:
// `ew` is the warp's number among them, row0 the first of its 32 rows; out_row0
// and out_col are where the tile's outputs go (bf16 modes: a split tile's copy
// has its own place and type).  wait() waits for the accumulator and is called
// after whatever can be loaded before it; it returns false after an abort.
template <int MODE, int TN, class Sh, class Wait, class Release>
__device__ __forceinline__ void epilogue_any(Sh &sh, int ew, int buf, uint32_t tbase, int row0, int out_row0,
                                             int tile_n, int out_col, int lane, const float *xs, bool has_bias, int M, int N,
                                             int out_f32, int swiglu, int tma_out, const CUtensorMap *tmOut,
                                             uint32_t &units_issued, void *out, int32_t *acc_out, const float *ws,
                                             const float *bias, const EpiArgs &ex, Wait wait, Release release)
{
    const int row = row0 + lane;
    const bool row_ok = row < M;
    const float *wsv = sh.wsb[buf], *bsv = sh.biasb[buf];
    constexpr int COLS = TN * 4 / epi_warps(MODE);  // the warp's columns of the tile
    const int c_lo = (ew >> 2) * COLS;
    if constexpr (!has_exponentials(MODE)) {
        if (!wait())
            return;
        float xm = 0.0f;
        bool live = row_ok;
        if constexpr (row_factor(MODE))
            live = row_ok && ex.takes_part(row, xm);
        else if constexpr (!is_bf16(MODE))
            xm = row_ok ? xs[row] : 0.0f;
        epilogue_tile<is_bf16(MODE), row_factor(MODE), MODE == kBf16RowsAdd, COLS>(
            tbase + (uint32_t)c_lo, out_row0, out_col + c_lo, lane, xm, live, wsv + c_lo, bsv + c_lo, has_bias, M, N,
            out_f32, swiglu, tma_out, tmOut, sh.epi[ew], units_issued, out, acc_out, ws, bias, release);
    } else {
        const int col_base = tile_n * TN;
        uint8_t *stage_buf = &sh.epi[0][0] + ew * (kEpiBytes / 2);
        const float xm = row_ok ? xs[row] : 0.0f;
        if constexpr (MODE == kSwigluGrad) {
            uint32_t dn[8];
            load_dout16(ex.dout + (int64_t)row * (N >> 1), (col_base + c_lo) >> 1, N >> 1, row_ok, dn);
            if (!wait())
                return;
            epilogue_swiglu_grad<COLS>(tbase, row0, col_base, c_lo, lane, xm, row_ok, wsv, bsv, has_bias, N, ex, tmOut,
                                 stage_buf, units_issued, dn, release);
        } else if constexpr (MODE == kCeGrad) {
            if (!wait())
                return;
            epilogue_ce_grad<COLS>(tbase, row0, col_base, c_lo, lane, xm, row_ok, wsv, bsv, has_bias, N, ex, tmOut,
                             stage_buf, units_issued, release);
        } else {
            // the two warps of a row join their halves: the upper one's pairs
            // go through its staging buffer (unused otherwise).  After an abort
            // both still meet at the barrier.
            const bool ok = wait();
            float2 a = make_float2(0.0f, 0.0f);
            if (ok)
                a = epilogue_ce_stats<COLS>(tbase, row, col_base, c_lo, xm, row_ok, wsv, bsv, has_bias, N, ex, release);
            float2 *half = reinterpret_cast<float2 *>(&sh.epi[0][0]) + 32 * (ew & 3);
            if (ew >= 4)
                half[lane] = a;
            asm volatile("bar.sync 3, 256;" ::: "memory");
            if (ok && ew < 4 && row_ok) {
                join(a, half[lane]);
                ex.part[(int64_t)row * ex.slices + ex.n0 / TN + tile_n] = a;
            }
        }
    }
}

// BF16 modes: A and B are bf16 (K counted in bf16 elements, 64 per 128-byte
// stage row), tcgen05.mma kind::f16 into fp32, and the epilogue writes the
// accumulators as they are (xs, ws, bias, swiglu and acc_out unused).
template <int MODE, int TN = BN>
__global__ void __launch_bounds__(threads(MODE), 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmCopy,
                const float *__restrict__ xs,
                const float *__restrict__ ws, const float *__restrict__ bias, int max_rows, int N, int K, int out_f32,
                int swiglu, int tma_out, void *__restrict__ out, int32_t *__restrict__ acc_out, const EpiArgs ex)
{
    constexpr bool BF16 = is_bf16(MODE);
    extern __shared__ uint8_t smem_raw[];
    using Sh = Smem<MODE, TN>;
    constexpr int kStages = Sh::kStages;
    Sh &sh = smem_aligned_1024<Sh>(smem_raw);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int BKE = BF16 ? BK / 2 : BK;  // K elements per stage
    const int kblocks = (K + BKE - 1) / BKE;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.tmem_full[b], 1);
            mbar_init(&sh.tmem_empty[b], epi_warps(MODE));
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, Sh::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (dependent(MODE)) {
        asm volatile("griddepcontrol.launch_dependents;" :::);
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    // the rows, known on the device only where ex.count is given
    int M = max_rows;
    if constexpr (dependent(MODE)) {
        if (ex.count != nullptr)
            M = min(M, __ldcg(ex.count));
    }
    const Tiling tiling(M, N, kblocks, BM, b_is_kn(MODE) ? ex.slots : 1, b_is_kn(MODE) ? ex.max_splits : 1,
                        b_is_kn(MODE) ? ex.split_tail : 0, TN);
    const int num_tiles = tiling.units;
    auto coords = [&](int unit, int &tm, int &tn, int &k0, int &k1, int &copy) {
        if constexpr (b_is_kn(MODE)) {
            return tiling.at(unit, tm, tn, k0, k1, copy);
        } else {
            if constexpr (dependent(MODE))
                tile_place(unit, tiling.tiles_m, tiling.tiles_n, tm, tn);
            else
                tile_coords(unit, tiling.tiles_n, tm, tn);
            k0 = 0;
            k1 = kblocks;
            copy = -1;
            return true;
        }
    };
    const uint32_t tmem = sh.tmem_base;
    volatile int *abort = &sh.abort;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            prefetch_tmap(&tmA);
            prefetch_tmap(&tmB);
            int stage = 0;
            uint32_t phase = 0;
            uint32_t issued = 0;  // stages filled so far
            bool ok = true;
            const uint32_t stage_bytes = (uint32_t)(Sh::kStageBytes - kABytes + a_box_rows(max_rows) * BK);
            for (int tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x) {
                int tm, tn, k0, k1, copy;
                if (!coords(tile, tm, tn, k0, k1, copy))
                    continue;
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait_bounded(&sh.empty[stage], phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sh.full[stage], stage_bytes);
                    tma_load_2d(sh.stage[stage], &tmA, kb * BKE, tm * BM, &sh.full[stage]);
                    if constexpr (b_is_kn(MODE)) {
#pragma unroll
                        for (int i = 0; i < TN / 64; ++i)  // boxes of 64 columns x 64 terms
                            tma_load_2d(sh.stage[stage] + kABytes + i * kKnBytes, &tmB, tn * TN + 64 * i, kb * BKE,
                                        &sh.full[stage]);
                    } else {
                        tma_load_2d(sh.stage[stage] + kABytes, &tmB, kb * BKE, tn * TN, &sh.full[stage]);
                    }
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // Let copies already in flight land before the CTA goes away.
                for (uint32_t s = 0; s < kStages && s < issued; ++s) {
                    volatile int no_abort = 0;
                    mbar_wait_bounded(&sh.full[s], ((issued - 1 - s) / kStages) & 1u, &no_abort, 20000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // The whole warp walks the loop, so that the descriptors stay in uniform
        // registers, where the MMA instruction takes them from; one lane issues.
        {
            const bool issuer = elect_one();
            int stage = 0;
            uint32_t phase = 0;
            int local = 0;
            bool ok = true;
            // descriptors of stage 0; 16 terms (32 bytes of a K-major row, 16 rows
            // of an MN-major box) on per MMA
            const uint32_t a_lo = sw128_kmajor_lo(smem_u32(sh.stage[0]));
            const uint32_t b_addr = smem_u32(sh.stage[0]) + kABytes;
            const uint32_t b_lo = b_is_kn(MODE) ? sw128_mnmajor_lo(b_addr, kKnBytes) : sw128_kmajor_lo(b_addr);
            constexpr uint32_t kBStep = b_is_kn(MODE) ? 2048 >> 4 : 32 >> 4;
            for (int tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x) {
                int tm, tn, k0, k1, copy;
                if (!coords(tile, tm, tn, k0, k1, copy))
                    continue;
                const int buf = local & 1;
                const uint32_t use = (uint32_t)(local >> 1) & 1u;
                if (!mbar_wait_bounded_warp(&sh.tmem_empty[buf], use ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * TN);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait_bounded_warp(&sh.full[stage], phase, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = (uint32_t)stage * (Sh::kStageBytes >> 4);
                    if (issuer) {
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk) {
                            const uint64_t ad = sw128_desc(a_lo + st + 2u * kk);
                            const uint64_t bd = sw128_desc(b_lo + st + kBStep * kk);
                            if constexpr (BF16)
                                mma_bf16(d, ad, bd, idesc_bf16(BM, TN, b_is_kn(MODE)), kk == 0 ? kb != k0 : 1u);
                            else
                                mma_i8(d, ad, bd, idesc_i8(BM, TN), kk == 0 ? kb != k0 : 1u);
                        }
                        tc_commit(&sh.empty[stage]);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok && issuer)
                    tc_commit(&sh.tmem_full[buf]);
                ++local;
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2..5, or 2..9)
        // Warp q owns TMEM lanes 32q..32q+31 = rows 32q.. of the tile.
        // Per tile: the epilogue threads stage the tile's channel scales
        // (and bias) in shared memory before waiting for the accumulator, so
        // that latency hides under the MMAs.  The accumulator is read 32
        // columns at a time, the next chunk's TMEM load in flight while the
        // current one is converted.  Fast path (tma_out): each 128-byte column
        // unit (64 bf16 or 32 fp32 columns) of the warp's 32 rows goes into a
        // 128B-swizzled staging buffer (16-byte chunk c of row r at chunk
        // c ^ (r % 8): conflict-free) and leaves with one TMA bulk store.  Otherwise (int32 accumulators requested, or rows
        // not 16-byte multiples) each thread stores its own row.
        // The loop never exits early: after an abort every warp still reaches
        // the same named barriers, skipping the work.
        const int q = warp & 3;
        const int et = threadIdx.x - 64;  // among the epilogue threads
        int local = 0;
        uint32_t units_issued = 0;
        for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
            int tm, tn, k0, k1, copy;
            if (!coords(tile, tm, tn, k0, k1, copy))
                continue;
            const int buf = local & 1;
            const uint32_t use = (uint32_t)(local >> 1) & 1u;
            ++local;
            if constexpr (!BF16) {
                for (int j = et; j < TN; j += 32 * epi_warps(MODE)) {
                    const int n = tn * TN + j, at = stage_column<MODE>(j);
                    sh.wsb[buf][at] = n < N ? ws[n] : 0.0f;
                    sh.biasb[buf][at] = (bias != nullptr && n < N) ? bias[n] : 0.0f;
                }
            }
            asm volatile("bar.sync 2, %0;" ::"n"(32 * epi_warps(MODE)) : "memory");
            auto wait = [&]() {
                const bool ok = mbar_wait_bounded_warp(&sh.tmem_full[buf], use, abort);
                tc_fence_after();
                return ok;
            };
            const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * TN);
            const int row0 = tm * BM + 32 * q;
            const bool whole = copy < 0;  // a whole tile: its outputs have their own place
            epilogue_any<MODE, TN>(sh, warp - 2, buf, tbase, row0, whole ? row0 : copy * BM + 32 * q, tn,
                               whole ? tn * TN : 0, lane, xs, bias != nullptr, M, N, whole ? out_f32 : 1, swiglu,
                               tma_out, whole ? &tmOut : &tmCopy, units_issued, out, acc_out, ws, bias, ex, wait, [&]() {
                              tc_fence_before();
                              __syncwarp();
                              if (lane == 0)
                                  mbar_arrive(&sh.tmem_empty[buf]);
                          });
        }
        if (lane == 0)
            bulk_wait_all();  // every output store has landed before the CTA exits
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Sh::kTmemCols);
    }
}


// ---------------------------------------------------------------- CTA-pair variant
//
// For problems with at least one 256 x 256 tile per SM pair: a cluster of two
// CTAs computes a 256 x 256 tile with tcgen05.mma.cta_group::2 (M = 256,
// N = 256, K = 32).  Each CTA loads only its own 128 rows of A and its own 128
// rows of B (no multicast loads), so every SM moves 32 KB instead of 48 KB per
// 128-wide K slice for the same MMA work; each CTA's TMEM receives its 128 rows
// of the accumulator.  The leader (rank 0) issues the MMAs; both CTAs' TMA
// copies signal the leader's "full" barrier; the leader's commits are sent to
// both CTAs' "empty" and "tmem_full" barriers; both CTAs' epilogue warps
// release the accumulator on the leader's "tmem_empty" barrier.
namespace pair {
constexpr int kStages = 6;
constexpr int kHalfBytes = 128 * BK;           // 16 KB: one CTA's half of A or of B
constexpr int kStageBytes = 2 * kHalfBytes;    // A half at +0, B half at +16 KB
constexpr uint32_t kIdesc = idesc_i8(256, BN);

template <int MODE>
struct __align__(1024) Smem {
    uint8_t stage[kStages][kStageBytes];
    uint8_t epi[epi_units(MODE)][kEpiBytes];
    float wsb[2][scale_cols(MODE, BN)];
    float biasb[2][scale_cols(MODE, BN)];
    uint64_t full[kStages];       // leader: both CTAs' bytes of a stage
    uint64_t empty[kStages];      // each CTA: its stage may be refilled
    uint64_t tmem_full[2];        // each CTA: its accumulator rows are complete
    uint64_t tmem_empty[2];       // leader: both CTAs' epilogues released the accumulator
    uint32_t tmem_base;
    int abort;
};
constexpr int kTmemCols = 2 * BN;  // two accumulators
template <int MODE>
constexpr size_t smem_bytes()
{
    static_assert(sizeof(Smem<MODE>) + 1024 <= kMaxSmem, "shared memory of one CTA");
    return sizeof(Smem<MODE>) + 1024;
}
}  // namespace pair

// BF16 as for gemm_kernel.
template <int MODE>
__global__ void __launch_bounds__(threads(MODE), 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmCopy,
                const float *__restrict__ xs,
                     const float *__restrict__ ws, const float *__restrict__ bias, int max_rows, int N, int K, int out_f32,
                     int swiglu, int tma_out, void *__restrict__ out, int32_t *__restrict__ acc_out, const EpiArgs ex)
{
    constexpr bool BF16 = is_bf16(MODE);
    extern __shared__ uint8_t smem_raw[];
    pair::Smem<MODE> &sh = smem_aligned_1024<pair::Smem<MODE>>(smem_raw);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int npairs = gridDim.x >> 1, pair_id = blockIdx.x >> 1;
    constexpr int BKE = BF16 ? BK / 2 : BK;  // K elements per stage
    const int kblocks = (K + BKE - 1) / BKE;
    if (threadIdx.x == 0) {
        for (int s = 0; s < pair::kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.tmem_full[b], 1);
            mbar_init(&sh.tmem_empty[b], 2 * epi_warps(MODE));
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc_pair(&sh.tmem_base, pair::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before anyone signals them
    tc_fence_after();
    if constexpr (dependent(MODE)) {
        asm volatile("griddepcontrol.launch_dependents;" :::);
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    // the rows, known on the device only where ex.count is given
    int M = max_rows;
    if constexpr (dependent(MODE)) {
        if (ex.count != nullptr)
            M = min(M, __ldcg(ex.count));
    }
    const Tiling tiling(M, N, kblocks, 256, b_is_kn(MODE) ? ex.slots : 1, b_is_kn(MODE) ? ex.max_splits : 1,
                        b_is_kn(MODE) ? ex.split_tail : 0);
    const int num_tiles = tiling.units;
    auto coords = [&](int unit, int &tm, int &tn, int &k0, int &k1, int &copy) {
        if constexpr (b_is_kn(MODE)) {
            return tiling.at(unit, tm, tn, k0, k1, copy);
        } else {
            if constexpr (dependent(MODE))
                tile_place(unit, tiling.tiles_m, tiling.tiles_n, tm, tn);
            else
                tile_coords(unit, tiling.tiles_n, tm, tn);
            k0 = 0;
            k1 = kblocks;
            copy = -1;
            return true;
        }
    };
    const uint32_t tmem = sh.tmem_base;
    volatile int *abort = &sh.abort;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            prefetch_tmap(&tmA);
            prefetch_tmap(&tmB);
            const uint32_t full0 = mapa_shared(smem_u32(&sh.full[0]), 0);  // the leader's
            const uint32_t pair_bytes = 2u * (uint32_t)(pair::kHalfBytes + a_box_rows(max_rows) * BK);
            int stage = 0;
            uint32_t phase = 0;
            uint32_t issued = 0;  // stages filled so far
            bool ok = true;
            for (int tile = pair_id; ok && tile < num_tiles; tile += npairs) {
                int tm, tn, k0, k1, copy;
                if (!coords(tile, tm, tn, k0, k1, copy))
                    continue;
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait_bounded(&sh.empty[stage], phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_leader = full0 + 8u * (uint32_t)stage;
                    if (leader)
                        mbar_arrive_expect_tx(&sh.full[stage], pair_bytes);
                    tma_load_2d_pair(sh.stage[stage], &tmA, kb * BKE, tm * 256 + (int)rank * 128, full_leader);
                    if constexpr (b_is_kn(MODE)) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)  // this CTA's 128 columns, in boxes of 64 columns x 64 terms
                            tma_load_2d_pair(sh.stage[stage] + pair::kHalfBytes + i * kKnBytes, &tmB,
                                             tn * BN + (int)rank * 128 + 64 * i, kb * BKE, full_leader);
                    } else {
                        tma_load_2d_pair(sh.stage[stage] + pair::kHalfBytes, &tmB, kb * BKE,
                                         tn * BN + (int)rank * 128, full_leader);
                    }
                    ++issued;
                    if (++stage == pair::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // let copies in flight land before the CTAs go away: the leader
                // waits on its barriers (bounded); the partner, whose copies
                // signal the leader, waits a fixed 100 us
                if (leader) {
                    for (uint32_t s = 0; s < pair::kStages && s < issued; ++s) {
                        volatile int no_abort = 0;
                        mbar_wait_bounded(&sh.full[s], ((issued - 1 - s) / pair::kStages) & 1u, &no_abort,
                                          20000000ull);
                    }
                } else {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 100000ull) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader only)
        if (leader) {  // the whole warp, as in gemm_kernel
            const bool issuer = elect_one();
            int stage = 0;
            uint32_t phase = 0;
            int local = 0;
            bool ok = true;
            // descriptors of stage 0; 16 terms (32 bytes of a K-major row, 16 rows
            // of an MN-major box) on per MMA
            const uint32_t a_lo = sw128_kmajor_lo(smem_u32(sh.stage[0]));
            const uint32_t b_addr = smem_u32(sh.stage[0]) + pair::kHalfBytes;
            const uint32_t b_lo = b_is_kn(MODE) ? sw128_mnmajor_lo(b_addr, kKnBytes) : sw128_kmajor_lo(b_addr);
            constexpr uint32_t kBStep = b_is_kn(MODE) ? 2048 >> 4 : 32 >> 4;
            for (int tile = pair_id; ok && tile < num_tiles; tile += npairs) {
                int tm, tn, k0, k1, copy;
                if (!coords(tile, tm, tn, k0, k1, copy))
                    continue;
                const int buf = local & 1;
                const uint32_t use = (uint32_t)(local >> 1) & 1u;
                if (!mbar_wait_bounded_warp(&sh.tmem_empty[buf], use ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * BN);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait_bounded_warp(&sh.full[stage], phase, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = (uint32_t)stage * (pair::kStageBytes >> 4);
                    if (issuer) {
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk) {
                            const uint64_t ad = sw128_desc(a_lo + st + 2u * kk);
                            const uint64_t bd = sw128_desc(b_lo + st + kBStep * kk);
                            if constexpr (BF16)
                                mma_bf16_pair(d, ad, bd, idesc_bf16(256, BN, b_is_kn(MODE)), kk == 0 ? kb != k0 : 1u);
                            else
                                mma_i8_pair(d, ad, bd, pair::kIdesc, kk == 0 ? kb != k0 : 1u);
                        }
                        tc_commit_both(smem_u32(&sh.empty[0]) + 8u * (uint32_t)stage);
                    }
                    if (++stage == pair::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok && issuer)
                    tc_commit_both(smem_u32(&sh.tmem_full[buf]));
                ++local;
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2..5, or 2..9, both CTAs)
        const int q = warp & 3;
        const int et = threadIdx.x - 64;
        int local = 0;
        uint32_t units_issued = 0;
        for (int tile = pair_id; tile < num_tiles; tile += npairs) {
            int tm, tn, k0, k1, copy;
            if (!coords(tile, tm, tn, k0, k1, copy))
                continue;
            const int buf = local & 1;
            const uint32_t use = (uint32_t)(local >> 1) & 1u;
            ++local;
            if constexpr (!BF16) {
                for (int j = et; j < BN; j += 32 * epi_warps(MODE)) {
                    const int n = tn * BN + j, at = stage_column<MODE>(j);
                    sh.wsb[buf][at] = n < N ? ws[n] : 0.0f;
                    sh.biasb[buf][at] = (bias != nullptr && n < N) ? bias[n] : 0.0f;
                }
            }
            asm volatile("bar.sync 2, %0;" ::"n"(32 * epi_warps(MODE)) : "memory");
            auto wait = [&]() {
                const bool ok = mbar_wait_bounded_warp(&sh.tmem_full[buf], use, abort);
                tc_fence_after();
                return ok;
            };
            const int row0 = tm * 256 + (int)rank * 128 + 32 * q;
            const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * BN);
            const uint32_t release_addr = mapa_shared(smem_u32(&sh.tmem_empty[buf]), 0);
            const bool whole = copy < 0;  // a whole tile: its outputs have their own place
            epilogue_any<MODE, BN>(sh, warp - 2, buf, tbase, row0, whole ? row0 : copy * 256 + (int)rank * 128 + 32 * q, tn,
                               whole ? tn * BN : 0, lane, xs, bias != nullptr, M, N, whole ? out_f32 : 1, swiglu,
                               tma_out, whole ? &tmOut : &tmCopy, units_issued, out, acc_out, ws, bias, ex, wait, [&]() {
                              tc_fence_before();
                              __syncwarp();
                              if (lane == 0)
                                  mbar_arrive_cluster(release_addr);
                          });
        }
        if (lane == 0)
            bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its partner may still signal it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, pair::kTmemCols);
    }
}

}  // namespace gm
}  // namespace cr

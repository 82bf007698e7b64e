// k_gemm_decode.cuh -- the int8 contraction of few rows on packed weights: the
// codes are decoded into the tensor core's operand stages, so the int8 weight is
// never stored.
//
//   acc[m, n] = sum_k xq[m, k] * w8[n, k]
//
// With one tile of 128 rows every weight is wanted by one CTA only, and decoding it
// to memory first (0.56 bytes read, 1 written, 1 read again) is most of the
// work.  Here a CTA owns TN = 128 columns (rows of the weight) at a time, or 64,
// with half the decoding warps, where there are few tiles:
//
//   warp 0       TMA of A's 128-term blocks into the operand ring
//   warp 1       tcgen05.mma kind::i8, 128 x TN tiles, two accumulators
//   warps 2..17  decode: codes, scales -> int8 in the operand ring's swizzled
//                layout (and, for a gradient, the bf16 weight to memory);
//                warps 2..9 do the tile's epilogue (k_gemm.cuh) after its last
//                block
//   warp 18      TMA of the codes and scales of 256 terms into their own ring
//
// Cross entropy of 17 x 131072 x 4096: 100 us (3.0 TB/s of codes and scales)
// against 219 with the weight decoded first; 128 rows 116 us; the gated gradient
// of 17 x 12288 x 4096 60 us against 73.  Bound by the latency of the decoding
// warps' chain (wait, two dependent shared-memory reads, decode, store, fence)
// and by shared memory (its pipe 62 % busy with the warps' accesses alone, beside
// the MMAs' operands and the copies; issue slots 51 %): 17 x 131072 x 4096 took
// 136 us with eight warps that handed over every block, 116 with two blocks at a
// time, 100 with sixteen warps.  Eight copies of the table (no bank conflicts,
// one slot of codes less) made no difference.
#pragma once

#include "cr_device.cuh"
#include "k_gemm.cuh"

namespace cr {
namespace gd {

constexpr int kStages = 4;       // operand ring, 128 terms each
constexpr int kRaw = 3;          // ring of packed codes, 256 terms each
constexpr int kLutCopies = 4;
constexpr int kWorkers = 256;    // threads of warps 2..9: the epilogue

// For tiles of TN columns.
template <int TN>
struct Sizes {
    static constexpr int kStageBytes = gm::kABytes + TN * gm::BK;
    static constexpr int kCodeBytes = TN * 64;   // codes of 128 terms
    static constexpr int kScaleBytes = TN * 16;  // scales of 256 terms
    static constexpr int kRawBytes = 2 * kCodeBytes + kScaleBytes;
    static constexpr int kDecoders = 4 * TN;     // threads from warp 2 on that decode
    static constexpr int kRawWarp = 2 + kDecoders / 32;
    static constexpr int kThreads = 32 * (kRawWarp + 1);
    static constexpr int kTmemCols = 2 * TN;
};

template <int MODE, int TN>
struct __align__(1024) Smem {
    uint8_t stage[kStages][Sizes<TN>::kStageBytes];
    uint8_t raw[kRaw][Sizes<TN>::kRawBytes];
    alignas(1024) uint8_t epi[gm::epi_units(MODE)][gm::kEpiBytes];
    uint4 lut[256 * kLutCopies];
    float wsb[2][TN];
    float biasb[2][TN];
    uint64_t full[kStages];      // A has landed and the decoding warps have written their parts of B
    uint64_t empty[kStages];
    uint64_t raw_full[kRaw];
    uint64_t raw_empty[kRaw];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint32_t tmem_base;
    int abort;
};

template <int MODE, int TN>
constexpr size_t smem_bytes()
{
    static_assert(sizeof(Smem<MODE, TN>) + 1024 <= gm::kMaxSmem, "shared memory of one CTA");
    return sizeof(Smem<MODE, TN>) + 1024;
}

// tmQ: qdata [N, K / 2] in boxes of 64 bytes x TN rows; tmS: srel [N, K / 16]
// in boxes of 16 bytes x TN rows; w: bf16 [N, K] to write, or null.
template <int MODE, int TN>
__global__ void __launch_bounds__(Sizes<TN>::kThreads, 1)
    gemm_decode_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmOut,
                       const float *__restrict__ codebook, const float *__restrict__ xs, const float *__restrict__ ws,
                       const float *__restrict__ bias, int M, int N, int K, uint16_t *__restrict__ w,
                       const gm::EpiArgs ex)
{
    extern __shared__ uint8_t smem_raw[];
    using S = Sizes<TN>;
    constexpr int kDecoders = S::kDecoders, kCodeBytes = S::kCodeBytes;
    Smem<MODE, TN> &sh = smem_aligned_1024<Smem<MODE, TN>>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kblocks = K / gm::BK, tiles_m = (M + gm::BM - 1) / gm::BM, tiles = (N + TN - 1) / TN * tiles_m;
    // tile t: rows 128 (t % tiles_m), columns TN (t / tiles_m)
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1 + kDecoders / 32);
            mbar_init(&sh.empty[s], 1);
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&sh.raw_full[s], 1);
            mbar_init(&sh.raw_empty[s], kDecoders / 32);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.tmem_full[b], 1);
            mbar_init(&sh.tmem_empty[b], kWorkers / 32);
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = sh.tmem_base;
    volatile int *abort = &sh.abort;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer of A
        if (lane == 0) {
            prefetch_tmap(&tmA);
            const uint32_t bytes = (uint32_t)(gm::a_box_rows(M) * gm::BK);
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x)
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded(&sh.empty[stage], phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sh.full[stage], bytes);
                    tma_load_2d(sh.stage[stage], &tmA, kb * gm::BK, tile % tiles_m * gm::BM, &sh.full[stage]);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            if (!ok) {
                // copies in flight land before the CTA goes away (nobody may
                // complete these barriers any more: the waits are bounded)
                for (uint32_t s = 0; s < kStages && s < issued; ++s) {
                    volatile int no_abort = 0;
                    mbar_wait_bounded(&sh.full[s], ((issued - 1 - s) / kStages) & 1u, &no_abort, 20000000ull);
                }
            }
        }
    } else if (warp == S::kRawWarp) {
        // ------------------------------------------------ TMA producer of codes and scales
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmS);
            int slot = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x)
                for (int kb = 0, n0 = tile / tiles_m * TN; kb < kblocks; kb += 2) {
                    if (!mbar_wait_bounded(&sh.raw_empty[slot], phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sh.raw_full[slot], S::kRawBytes);
                    tma_load_2d(sh.raw[slot], &tmQ, kb * 64, n0, &sh.raw_full[slot]);
                    tma_load_2d(sh.raw[slot] + kCodeBytes, &tmQ, kb * 64 + 64, n0, &sh.raw_full[slot]);
                    tma_load_2d(sh.raw[slot] + 2 * kCodeBytes, &tmS, kb * 8, n0, &sh.raw_full[slot]);
                    ++issued;
                    if (++slot == kRaw) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            if (!ok) {
                for (uint32_t s = 0; s < kRaw && s < issued; ++s) {
                    volatile int no_abort = 0;
                    mbar_wait_bounded(&sh.raw_full[s], ((issued - 1 - s) / kRaw) & 1u, &no_abort, 20000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (the whole warp, as in gemm_kernel)
        const bool issuer = elect_one();
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t a_lo = sw128_kmajor_lo(smem_u32(sh.stage[0]));
        const uint32_t b_lo = sw128_kmajor_lo(smem_u32(sh.stage[0]) + gm::kABytes);
        for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, ++local) {
            const int buf = local & 1;
            if (!mbar_wait_bounded_warp(&sh.tmem_empty[buf], ((uint32_t)(local >> 1) & 1u) ^ 1u, abort))
                break;
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(buf * TN);
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!mbar_wait_bounded_warp(&sh.full[stage], phase, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = (uint32_t)stage * (S::kStageBytes >> 4);
                if (issuer) {
#pragma unroll
                    for (int kk = 0; kk < gm::BK / 32; ++kk)
                        mma_i8(d, sw128_desc(a_lo + st + 2u * kk), sw128_desc(b_lo + st + 2u * kk),
                               idesc_i8(gm::BM, TN), kk == 0 ? kb != 0 : 1u);
                    tc_commit(&sh.empty[stage]);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok && issuer)
                tc_commit(&sh.tmem_full[buf]);
        }
    } else {
        // ------------------------------------------------ decode (warps 2..17), then epilogue (warps 2..9)
        const int et = threadIdx.x - 64, q = warp & 3;
        {
            const uint4 e = lut_entry((uint32_t)et & 255u, codebook);
#pragma unroll
            for (int c = et >> 8; c < kLutCopies; c += kDecoders / 256)
                sh.lut[(et & 255) * kLutCopies + c] = e;
        }
        asm volatile("bar.sync 4, %0;" ::"n"(kDecoders) : "memory");
        const uint4 *lut = sh.lut + (et & (kLutCopies - 1));
        // items of 32 weights of a 128-term block: row it / 4, quarter it % 4 (two
        // 16-byte chunks of the operand); a thread has kItems of each block
        constexpr int kItems = TN * 4 / kDecoders;
        int stage = 0, slot = 0, local = 0;
        uint32_t phase = 0, raw_phase = 0;
        uint32_t units_issued = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++local) {
            const int tn = tile / tiles_m, row_base = tile % tiles_m * gm::BM;
            float sc[kItems];
            if constexpr (MODE != gm::kCeStats) {
#pragma unroll
                for (int u = 0; u < kItems; ++u) {
                    const int n = tn * TN + ((et + kDecoders * u) >> 2);
                    sc[u] = n < N ? __bfloat162float(__float2bfloat16_rn(ws[n])) : 0.0f;
                }
            }
            for (int kb = 0; ok && kb < kblocks; kb += 2) {  // 256 terms: one slot of the raw ring, two stages
                ok = mbar_wait_bounded_warp(&sh.raw_full[slot], raw_phase, abort) &&
                     mbar_wait_bounded_warp(&sh.empty[stage], phase ^ 1u, abort) &&
                     mbar_wait_bounded_warp(&sh.empty[stage + 1], phase ^ 1u, abort);
                if (!ok)
                    break;
                const uint8_t *raw = sh.raw[slot];
                uint4 c[2 * kItems];
                uint32_t s[2 * kItems];
#pragma unroll
                for (int u = 0; u < 2 * kItems; ++u) {
                    const int half = u / kItems, it = et + kDecoders * (u % kItems);
                    c[u] = *reinterpret_cast<const uint4 *>(raw + half * kCodeBytes + 16 * it);
                    s[u] = *reinterpret_cast<const uint16_t *>(raw + 2 * kCodeBytes + 16 * (it >> 2) + 8 * half +
                                                               2 * (it & 3));
                }
#pragma unroll
                for (int u = 0; u < 2 * kItems; ++u) {
                    const int half = u / kItems, it = et + kDecoders * (u % kItems), row = it >> 2, part = it & 3;
                    uint8_t *b = sh.stage[stage + half] + gm::kABytes + 128 * row;
                    const uint32_t code[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint4 T = lut[kLutCopies * ((s[u] >> (8 * g)) & 0xFFu)];
                        uint32_t o[4];
                        decode8(code[2 * g], T, o[0], o[1]);
                        decode8(code[2 * g + 1], T, o[2], o[3]);
                        *reinterpret_cast<uint4 *>(b + 16 * ((2 * part + g) ^ (row & 7))) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                        if constexpr (MODE != gm::kCeStats) {
                            const int n = tn * TN + row;
                            if (n < N && row_base == 0)  // the first tile of rows writes the weight
                                store_bf16_weights(w + (int64_t)n * K + (kb + half) * gm::BK + 32 * part + 16 * g, o,
                                                   sc[u % kItems]);
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.full[stage]);
                    mbar_arrive(&sh.full[stage + 1]);
                    mbar_arrive(&sh.raw_empty[slot]);
                }
                if ((stage += 2) == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++slot == kRaw) {
                    slot = 0;
                    raw_phase ^= 1u;
                }
            }
            if (kDecoders > kWorkers && et >= kWorkers)
                continue;
            const int buf = local & 1;
            const uint32_t use = (uint32_t)(local >> 1) & 1u;
            if (et < TN) {
                const int n = tn * TN + et, at = gm::stage_column<MODE>(et);
                sh.wsb[buf][at] = n < N ? ws[n] : 0.0f;
                sh.biasb[buf][at] = (bias != nullptr && n < N) ? bias[n] : 0.0f;
            }
            asm volatile("bar.sync 2, %0;" ::"n"(kWorkers) : "memory");
            const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * TN);
            auto wait = [&]() {
                ok = ok && mbar_wait_bounded_warp(&sh.tmem_full[buf], use, abort);
                tc_fence_after();
                return ok;
            };
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.tmem_empty[buf]);
            };
            const int row0 = row_base + 32 * q;
            if (row0 < M) {
                gm::epilogue_any<MODE, TN>(sh, warp - 2, buf, tbase, row0, row0, tn, tn * TN, lane, xs,
                                           bias != nullptr, M, N, 0, 0, 1, &tmOut, units_issued, nullptr, nullptr, ws,
                                           bias, ex, wait, release);
            } else {  // none of the warp's rows exists
                if (wait())
                    release();
                if constexpr (MODE == gm::kCeStats)
                    asm volatile("bar.sync 3, 256;" ::: "memory");  // as in epilogue_any
            }
        }
        if (lane == 0)
            bulk_wait_all();  // every output store has landed before the CTA exits
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmemCols);
    }
}

}  // namespace gd
}  // namespace cr

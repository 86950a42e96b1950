// fp4_gemm_pair.cuh -- the product of microscaled 4-bit matrices for more
// tokens: two SMs work on one tile (tcgen05 cta_group::2).
//
// A pair of CTAs holds a tile of 256 tokens x BT weight rows: each CTA the
// accumulators of its 128 tokens, in its shared memory the codes of those
// tokens and of half the weight rows (the tensor cores read the other half
// from the peer), and the scales of its tokens and of all BT weight rows.  So
// a 256-k stage of a 256 x 256 tile brings 38 KB to an SM for 512 cycles of
// MMAs; a tile of one SM would bring as much for half the work, more than an
// SM can load from L2.
//   Persistent: pairs take tiles in turn, tokens fastest, so that the pairs at
// work share weight rows in L2.  Warp 0 of each CTA loads its part of a stage
// and completes on the first CTA's barrier; warp 1 of the first CTA issues the
// scale copies and MMAs of both; eight epilogue warps per CTA empty the
// accumulators into registers as 16-bit values, release them and store rows
// while the next tile runs (two accumulators where they fit: BT <= 128).
#pragma once

#include "fp4_gemm.cuh"

namespace bitnet {

constexpr int kFp4PairEpiWarps = 8;
constexpr int kFp4PairThreads = 64 + 32 * kFp4PairEpiWarps;

struct Fp4PairArgs {
    int64_t M, N, K, ldy;
    const float *ga, *gw;
    void *y;
    int ytype;
    int tiles_m, tiles_n;  // 256-token and BT-row tiles
    int vec;               // rows of y start on 32-byte boundaries
};

template <int FMT, int BT>
struct Fp4Pair {
    static constexpr int kTiles = FMT == BITNET_FP4_MX ? 2 : 4;  // scale tiles per stage and 128 rows
    static constexpr int kBands = (BT + 127) / 128;              // 128-row bands of weight scales
    static constexpr int kAcc = BT <= 128 ? 2 : 1;               // accumulators
    static constexpr int kABytes = 128 * 128, kWBytes = BT / 2 * 128, kS = kTiles * kFp4TileBytes;
    static constexpr int kStage = kABytes + kWBytes + (1 + kBands) * kS;
    static constexpr int kOut = kFp4PairEpiWarps * 32 * 17 * 4;  // per-warp transposition of ragged outputs
    static constexpr int kStages = (222 * 1024 - kOut) / kStage < 8 ? (222 * 1024 - kOut) / kStage : 8;
    static constexpr int kOutAt = kStages * kStage;
    static constexpr int kBars = kOutAt + kOut;
    static constexpr int kBytes = kBars + (2 * kStages + 5) * 8 + 16;
    static constexpr int kSlotCols = 4 * kTiles * (1 + kBands);  // tensor-memory columns of a stage's scales
    static constexpr int kNeed = kAcc * BT + 2 * kSlotCols;
    static constexpr int kCols = kNeed <= 256 ? 256 : 512;
    static_assert(kNeed <= 512 && kStages >= 3 && BT % 64 == 0 && BT <= 256, "tile");
    static_assert(kStage % 1024 == 0 && kWBytes % 1024 == 0, "swizzled rows");
};

// A TMA load of one CTA of a pair that completes on a barrier of either (an
// address in the cluster's shared memory).
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int FMT>
__device__ __forceinline__ void umma_fp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                              uint32_t sb, uint32_t accumulate) {
    if (FMT == BITNET_FP4_MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// Each CTA of the pair copies the tile at this offset of its own shared memory.
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint32_t saddr) {
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrives on the barrier at this offset in both CTAs once the tensor-core work
// issued so far is done.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Two fp32 values as 16-bit ones, a in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
    uint32_t r;
    if (dtype == BITNET_FP16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ void stg_32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <int FMT, int BT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp4PairThreads, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                    const __grid_constant__ CUtensorMap samap, const __grid_constant__ CUtensorMap swmap,
                    const Fp4PairArgs a) {
    using L = Fp4Pair<FMT, BT>;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::kBars);  // of the first CTA: both CTAs' bytes
    uint64_t *empty = full + S;                                   // of each CTA
    uint64_t *acc_full = empty + S;                               // [2], of each CTA
    uint64_t *acc_empty = acc_full + 2;                           // [2], of the first CTA
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int units = a.tiles_m * a.tiles_n;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int64_t kp = k_pad(a.K);
    const int nk = (int)ceil_div(kp, kFp4StageK);
    const int tiles = (int)fp4_scale_tiles(a.K, FMT);

    if (threadIdx.x == 0) {
        prefetch_tensormap(&amap);
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&samap);
        prefetch_tensormap(&swmap);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(&acc_full[d], 1);
            mbar_init(&acc_empty[d], 2 * kFp4PairEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(L::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            int g = 0;  // stages over all of this pair's tiles
            bool ok = true;
            for (int u = pair; ok && u < units; u += pairs) {
                const int tm = u % a.tiles_m, tn = u / a.tiles_m;
                const int m0 = tm * 256 + (int)rank * 128;
                const int64_t n0 = (int64_t)tn * BT;
                for (int i = 0; i < nk; ++i, ++g) {
                    const int s = g % S;
                    if (g >= S && !tc_wait(&empty[s], (uint32_t)(g / S - 1) & 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = sm + s * L::kStage;
                    const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
                    tma_load_pair(st, &amap, i * 128, m0, bar);
                    tma_load_pair(st + L::kABytes, &wmap, i * 128, (int)(n0 + rank * (BT / 2)), bar);
                    uint8_t *ss = st + L::kABytes + L::kWBytes;
                    tma_load_pair(ss, &samap, 0, (m0 / 128) * tiles + i * L::kTiles, bar);
#pragma unroll
                    for (int b = 0; b < L::kBands; ++b)
                        tma_load_pair(ss + (1 + b) * L::kS, &swmap, 0, (int)(n0 / 128 + b) * tiles + i * L::kTiles, bar);
                }
            }
            // no copy may still be landing when the pair leaves (the first CTA
            // sees both CTAs' copies; they leave together)
            if (rank == 0)
                for (int j = g - S < 0 ? 0 : g - S; j < g; ++j) mbar_wait_bounded(&full[j % S], (uint32_t)(j / S) & 1u);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0 && lane == 0) {
            constexpr uint32_t idesc = fp4_idesc(FMT, 256, BT);
            bool ok = true;
            int g = 0, li = 0;
            for (int u = pair; ok && u < units; u += pairs, ++li) {
                const int d = li % L::kAcc;
                if (li >= L::kAcc && !tc_wait(&acc_empty[d], (uint32_t)(li / L::kAcc - 1) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dt = tmem + (uint32_t)(d * BT);
                // a 64-row tile starts in the middle of a 128-row band
                const uint32_t off = (uint32_t)(((int64_t)(u / a.tiles_m) * BT % 128) / 32);
                for (int i = 0; i < nk; ++i, ++g) {
                    const int s = g % S;
                    if (!tc_wait(&full[s], (uint32_t)(g / S) & 1u, abort_flag) ||
                        (g >= 2 && !tc_wait(&empty[(g - 2) % S], (uint32_t)((g - 2) / S) & 1u, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t aa = smem_u32(sm + s * L::kStage), wa = aa + L::kABytes;
                    const uint32_t saa = wa + L::kWBytes, swa = saa + L::kS;
                    const uint32_t ca = tmem + (uint32_t)(L::kAcc * BT + (g & 1) * L::kSlotCols), cw = ca + 4 * L::kTiles;
                    const int64_t left = (kp - (int64_t)i * kFp4StageK) / 64;
                    const int steps = (int)(left < 4 ? left : 4);
#pragma unroll
                    for (int t = 0; t < L::kTiles; ++t) {
                        tmem_cp_scales_pair(ca + 4 * t, saa + t * kFp4TileBytes);
#pragma unroll
                        for (int b = 0; b < L::kBands; ++b)
                            tmem_cp_scales_pair(cw + 4 * (t * L::kBands + b), swa + b * L::kS + t * kFp4TileBytes);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j < steps) {
                            const int t = FMT == BITNET_FP4_MX ? j >> 1 : j;
                            const int id = FMT == BITNET_FP4_MX ? (j & 1) * 2 : 0;
                            umma_fp4_pair<FMT>(dt, umma_desc_sw128(aa + 32 * j), umma_desc_sw128(wa + 32 * j),
                                               idesc | fp4_scale_id(id), ca + 4 * t, cw + 4 * t * L::kBands + off,
                                               (i > 0 || j > 0) ? 1u : 0u);
                        }
                    }
                    umma_commit_pair(&empty[s]);
                }
                if (ok) umma_commit_pair(&acc_full[d]);
            }
            if (!ok) {
                umma_commit_pair(drain);  // the MMAs issued so far end before tensor memory is freed
                mbar_wait_bounded(drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- epilogue
        constexpr int kCw = BT / 2;  // columns per warp: two warps share a lane quarter
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * kCw);
        uint32_t *buf = reinterpret_cast<uint32_t *>(sm + L::kOutAt) + (warp - 2) * 32 * 17;
        const float gs = (a.ga != nullptr ? *a.ga : 1.0f) * (a.gw != nullptr ? *a.gw : 1.0f);
        int li = 0;
        for (int u = pair; u < units; u += pairs, ++li) {
            const int d = li % L::kAcc;
            if (!__all_sync(0xffffffffu, tc_wait(&acc_full[d], (uint32_t)(li / L::kAcc) & 1u, abort_flag))) break;
            tc_fence_after();
            // 64 columns at a time, kept as 16-bit pairs
            uint32_t v[kCw / 2];
#pragma unroll
            for (int c0 = 0; c0 < kCw; c0 += 64) {
                uint32_t f[kCw < 64 ? kCw : 64];
#pragma unroll
                for (int c = 0; c < kCw - c0 && c < 64; c += 32) tmem_ld32(t0 + (uint32_t)(d * BT + c0 + c), f + c);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < kCw - c0 && c < 64; c += 2)
                    v[(c0 + c) / 2] =
                        pack2(__fmul_rn(__uint_as_float(f[c]), gs), __fmul_rn(__uint_as_float(f[c + 1]), gs), a.ytype);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&acc_empty[d]), 0));
            const int tm = u % a.tiles_m;
            const int64_t m0 = (int64_t)tm * 256 + rank * 128 + quarter * 32, n0 = (int64_t)(u / a.tiles_m) * BT + half * kCw;
            if (a.vec && n0 + kCw <= a.N) {
                uint16_t *yp = static_cast<uint16_t *>(a.y) + (m0 + lane) * a.ldy + n0;
                if (m0 + lane < a.M) {
#pragma unroll
                    for (int c = 0; c < kCw; c += 16) stg_32(yp + c, v + c / 2);
                }
            } else {
                // through shared memory, so that a store covers 32 columns of a row
#pragma unroll
                for (int c = 0; c < kCw; c += 32) {
                    __syncwarp();
#pragma unroll
                    for (int w = 0; w < 16; ++w) buf[lane * 17 + w] = v[c / 2 + w];
                    __syncwarp();
                    const int64_t n = n0 + c + lane;
                    for (int r = 0; r < 32; ++r)
                        if (m0 + r < a.M && n < a.N)
                            static_cast<uint16_t *>(a.y)[(m0 + r) * a.ldy + n] =
                                reinterpret_cast<const uint16_t *>(buf + r * 17)[lane];
                }
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA signals the other or reads its shared memory any more
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
}

}  // namespace bitnet

// fp4_gemm_pair.cuh -- the product of microscaled 4-bit matrices for more
// tokens: two SMs work on one tile (tcgen05 cta_group::2).
//
// A pair of CTAs holds a tile of 256 tokens x BT weight rows: each CTA the
// accumulators of its 128 tokens, in its shared memory the codes of those
// tokens and of half the weight rows (the tensor cores read the other half
// from the peer), and the scales of its tokens and of all BT weight rows.
//   What bounds it: an SM takes in some 64 bytes a cycle from L2, and a 256-k
// stage (16 KB of token codes, 64 BT bytes of weight codes, the scales) feeds
// 2 BT cycles of MMAs.  64 to 192 rows are bound by the loads (352 to 483
// cycles a stage), 384 rows by the MMAs (768).  Tiles of more than 192 rows are
// multiplied in two halves with an accumulator each from the same token codes.
//   Persistent: pairs take tiles in turn, tokens fastest, so that the pairs at
// work share weight rows in L2.  Warp 0 of each CTA loads its part of a stage
// and completes on the first CTA's barrier; warp 1 of the first CTA issues the
// scale copies and MMAs of both; eight epilogue warps per CTA empty the
// accumulators into registers, release them one by one and store rows while
// the next tile runs (up to 192 rows it runs in the other accumulator, above
// that the first half's MMAs run while the second half is emptied).
#pragma once

#include <type_traits>

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
    int split;             // SPLIT: pairs to a tile, in one cluster
    int test_stall;        // the first pair never asks for its first stage (test of the bounded waits)
};

template <int FMT, int BT>
struct Fp4Pair {
    static constexpr int kTiles = FMT == BITNET_FP4_MX ? 2 : 4;  // scale tiles per stage and 128 rows
    // A tile starts on a multiple of 64 rows, and so does its second half, so their weight scales may start in the
    // middle of a 128-row band: two tensor-memory columns in.  (An odd column, as tiles of 96 or 160 rows would need,
    // is refused by the MMA.)
    static constexpr int kBands = (BT + 127) / 128;
    static constexpr int kHalves = BT > 192 ? 2 : 1;
    static constexpr int kCols = BT / kHalves;                   // columns of an accumulator; there are two
    static constexpr int kABytes = 128 * 128, kWBytes = BT / 2 * 128, kS = kTiles * kFp4TileBytes;
    static constexpr int kStage = kABytes + kWBytes + (1 + kBands) * kS;
    static constexpr int kOut = kFp4PairEpiWarps * 4096;         // a box of 32 rows x 128 bytes of y per warp
    // Tensor-memory columns of a stage's scales, and how many stages' fit beside the accumulators.  With as many as
    // shared-memory stages, a stage's columns are free when its codes are; with fewer (two, for 192 and 384 rows of NV)
    // the issuer also waits for older MMAs, some 90 cycles a stage (which 384 rows' 768 cycles hide).  So no more
    // shared-memory stages than that, unless it leaves fewer than four.
    static constexpr int kSlotCols = 4 * kTiles * (1 + kBands);
    static constexpr int kFit = (512 - 2 * kCols) / kSlotCols;
    static constexpr int kMost = kFit >= 4 && kFit < 8 ? kFit : 8;
    static constexpr int kStages = (225 * 1024 - kOut) / kStage < kMost ? (225 * 1024 - kOut) / kStage : kMost;
    static constexpr int kOutAt = kStages * kStage;
    static constexpr int kBars = kOutAt + kOut;
    static constexpr int kBytes = kBars + (2 * kStages + 5) * 8 + 16;
    static constexpr int kSlots = kFit < kStages ? kFit : kStages;
    static constexpr int kNeed = 2 * kCols + kSlots * kSlotCols;
    static constexpr int kTmem = kNeed <= 256 ? 256 : 512;
    static_assert(kNeed <= 512 && kStages >= 3 && kSlots >= 2 && kCols % 64 == 0 && kCols <= 192, "tile");
    static_assert(kHalves == 1 || BT % 128 == 0, "whole bands");
    static_assert(kStage % 1024 == 0 && kCols / 2 * 128 % 1024 == 0, "swizzled rows");
    static_assert(kBytes + 1024 <= 232448, "shared memory");
    static_assert(BT > 128 || 128 * (BT * 4 + 16) <= kOutAt, "sums of a split tile take the stages' place");
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
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrives on the barrier at this offset in both CTAs (or the first alone; `lead`
// is its cluster rank) once the tensor-core work issued so far is done.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar, uint32_t lead, uint32_t ctas = 3u) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)(ctas << lead))
        : "memory");
}

// Arrives on a barrier of either CTA.  Release order at CTA scope is enough: what
// it tells the other CTA is that tensor memory has been read (tcgen05.wait::ld
// and the fence before), no memory; at cluster scope the arrival took 1000 to
// 1700 cycles.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    if (DT == BITNET_FP16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Sums times both factors as 16-bit pairs.  PACKED: packed multiplications, as
// many instructions as one factor takes unpacked (2048 x 13824 x 2560 MX, 384
// rows: 35.3 us; with a branch around the second factor 36.4).  Up to 192 rows
// that branch is the shorter way (512 x 6912 x 2560 NV: 7.47 us, packed 7.60).
template <int DT, bool PACKED, int N>
__device__ __forceinline__ void pack_all(uint32_t (&v)[N], uint32_t (&f)[2 * N], float2 g) {
    float last = g.x;
    if (!PACKED && __builtin_expect(g.y != 1.0f, 0)) {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) f[i] = __float_as_uint(__fmul_rn(__uint_as_float(f[i]), g.x));
        last = g.y;
    }
    const uint64_t g0 = f2_pack(g.x, g.x), g1 = f2_pack(g.y, g.y);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float s0 = __uint_as_float(f[2 * i]), s1 = __uint_as_float(f[2 * i + 1]);
        const float2 t = PACKED ? f2_unpack(f2_mul(f2_mul(f2_pack(s0, s1), g0), g1))
                                : make_float2(__fmul_rn(s0, last), __fmul_rn(s1, last));
        v[i] = pack2<DT>(t.x, t.y);
    }
}

// Stores 8 * pieces columns (64 or 32) of a warp's 32 rows, a lane's row as the
// 16-bit pairs v[at], v[at + 1], ...: put down as 128-byte rows of shared memory
// (16-byte piece w of row r at piece w ^ (r % 8), so that neither the lanes'
// rows nor a row's pieces share banks) and stored from there, whole rows of
// lines at a time.
//   Rows of y off 16-byte boundaries are stored as the 4-byte words that lie on
// 4-byte boundaries of y: a lane whose row starts between two puts its pairs
// down shifted by one value, and stores the row's first and last value itself.
// (2047 x 13823 x 2560 MX takes 40 us; 55 where each lane puts its words
// together from two reads.)
template <bool VEC, int N>
__device__ __forceinline__ void store_box(const Fp4PairArgs &a, uint8_t *box, const uint32_t (&v)[N], int at, int pieces,
                                          uint16_t *y, int rows, int64_t nb, int lane) {
    const int width = 8 * pieces;
    const int cols = (int)(a.N - nb < width ? (a.N - nb < 0 ? 0 : a.N - nb) : width);
    // whether row r of y starts between two 4-byte words: first_odd + r * step_odd is odd
    const int first_odd = VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(y + nb) >> 1 & 1);
    const int step_odd = VEC ? 0 : (int)(a.ldy & 1);
    __syncwarp();  // the rows of the last box have been read
    if (VEC || (first_odd | step_odd) == 0) {
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (at + 4 * w >= N) break;
            *reinterpret_cast<uint4 *>(box + lane * 128 + ((w ^ (lane & 7)) << 4)) =
                make_uint4(v[at + 4 * w], v[at + 4 * w + 1], v[at + 4 * w + 2], v[at + 4 * w + 3]);
        }
    } else {
        const bool odd = (first_odd + lane * step_odd) & 1;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (at + 4 * w >= N) break;
            uint32_t t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = at + 4 * w + i;
                t[i] = odd ? __funnelshift_l(j > at ? v[j - 1] : 0u, v[j], 16) : v[j];
            }
            *reinterpret_cast<uint4 *>(box + lane * 128 + ((w ^ (lane & 7)) << 4)) = make_uint4(t[0], t[1], t[2], t[3]);
        }
        if (odd && lane < rows) {
            uint16_t *yr = y + lane * a.ldy + nb;
            if (cols > 0) yr[0] = (uint16_t)v[at];
            if (cols == 64 && at + 31 < N) yr[63] = (uint16_t)(v[at + 31 < N ? at + 31 : 0] >> 16);
            if (cols == 32 && pieces == 4) yr[31] = (uint16_t)(v[at + 15] >> 16);
        }
    }
    __syncwarp();
    if constexpr (VEC) {
        const int w = lane & (pieces - 1), step = 32 / pieces;
        const int64_t n = nb + 8 * w;
        if (rows == 32 && cols == width) {  // a whole box: every row is read before the first is stored
            auto whole = [&](auto p) {
                constexpr int kPieces = decltype(p)::value, kStep = 32 / kPieces;
                uint4 t[kPieces];
                const int r0 = lane / kPieces;
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    t[i] = *reinterpret_cast<const uint4 *>(box + (r0 + kStep * i) * 128 + ((w ^ ((r0 + kStep * i) & 7)) << 4));
#pragma unroll
                for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4 *>(y + (r0 + kStep * i) * a.ldy + n) = t[i];
            };
            if (pieces == 8)
                whole(std::integral_constant<int, 8>{});
            else
                whole(std::integral_constant<int, 4>{});
            return;
        }
        for (int r = lane / pieces; r < rows; r += step) {
            const uint4 t = *reinterpret_cast<const uint4 *>(box + r * 128 + ((w ^ (r & 7)) << 4));
            uint16_t *yp = y + r * a.ldy + n;
            if (n + 8 <= a.N) {
                *reinterpret_cast<uint4 *>(yp) = t;
            } else {
                const uint32_t q[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < a.N) yp[e] = (uint16_t)(q[e >> 1] >> (16 * (e & 1)));
            }
        }
    } else {
        if (lane >= width / 2) return;
        if (rows == 32 && cols == width) {  // a whole box: even and odd rows each have their shift, pointer and lanes
            const int odd0 = first_odd, odd1 = (first_odd + step_odd) & 1;
            const bool go0 = lane > 0 || !odd0, go1 = lane > 0 || !odd1;
            uint16_t *y0 = y + nb + 2 * lane - odd0, *y1 = y + nb + 2 * lane - odd1 + a.ldy;
            const int64_t step = 2 * a.ldy;
            const uint8_t *from = box + 4 * (lane & 3);
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {  // eight rows are read before the first is stored
                uint32_t t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t[i] = *reinterpret_cast<const uint32_t *>(from + (r0 + i) * 128 + (((lane >> 2) ^ i) << 4));
#pragma unroll
                for (int i = 0; i < 8; i += 2, y0 += step, y1 += step) {
                    if (go0) *reinterpret_cast<uint32_t *>(y0) = t[i];
                    if (go1) *reinterpret_cast<uint32_t *>(y1) = t[i + 1];
                }
            }
            return;
        }
        const uint8_t *br = box + 4 * (lane & 3);
        uint16_t *yr = y + nb + 2 * lane;
        for (int r0 = 0; r0 < rows; r0 += 8, br += 1024, yr += 8 * a.ldy) {
            uint32_t t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = *reinterpret_cast<const uint32_t *>(br + i * 128 + (((lane >> 2) ^ i) << 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (r0 + i >= rows) break;
                const int shift = (first_odd + i * step_odd) & 1, e = 2 * lane - shift;
                uint16_t *p = yr + i * a.ldy - shift;
                if (e >= 0 && e + 1 < cols)
                    *reinterpret_cast<uint32_t *>(p) = t[i];
                else if (e >= 0 && e < cols)
                    p[0] = (uint16_t)t[i];
            }
        }
    }
}

// VEC: rows of y start on 16-byte boundaries.  SPLIT: for few tiles over a long
// k, a.split pairs share a tile (a cluster, and no tile after it): each sums a
// range of k, puts its sums into its stages' place and, once all have, adds up
// and stores its share of the rows, in the pairs' order.
template <int FMT, int BT, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(kFp4PairThreads, 1)
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
    const uint32_t lead = cluster_rank() & ~1u, rank = cluster_rank() & 1u;  // the pair's first CTA, and which this is
    const int units = a.tiles_m * a.tiles_n;
    const int pair = SPLIT ? (int)blockIdx.x / (2 * a.split) : blockIdx.x >> 1, pairs = SPLIT ? units : gridDim.x >> 1;
    const int64_t kp = k_pad(a.K);
    const int stages = (int)ceil_div(kp, kFp4StageK);
    const int part_k = (int)lead >> 1;  // SPLIT: the pair in its cluster
    const int k0 = SPLIT ? (int)((int64_t)stages * part_k / a.split) : 0;
    const int nk = SPLIT ? (int)((int64_t)stages * (part_k + 1) / a.split) : stages;  // this pair's stages: k0 .. nk - 1
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
                     "r"(L::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();  // both CTAs' barriers are set up (and fenced)
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        int g = 0;  // stages over all of this pair's tiles
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const int tm = u % a.tiles_m, tn = u / a.tiles_m;
            const int m0 = tm * 256 + (int)rank * 128;
            const int64_t n0 = (int64_t)tn * BT;
            for (int i = k0; i < nk; ++i, ++g) {
                const int s = g % S;
                if (g >= S && !warp_wait(&empty[s], (uint32_t)(g / S - 1) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                if (a.test_stall && pair == 0 && g == 0) continue;
                if (elect_one()) {
                    uint8_t *st = sm + s * L::kStage;
                    const uint32_t bar = map_rank(smem_u32(&full[s]), lead);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
                    tma_load_pair(st, &amap, i * 128, m0, bar);
#pragma unroll
                    for (int h = 0; h < L::kHalves; ++h)
                        tma_load_pair(st + L::kABytes + h * (L::kCols / 2 * 128), &wmap, i * 128,
                                      (int)(n0 + h * L::kCols + rank * (L::kCols / 2)), bar);
                    uint8_t *ss = st + L::kABytes + L::kWBytes;
                    tma_load_pair(ss, &samap, 0, (m0 / 128) * tiles + i * L::kTiles, bar);
#pragma unroll
                    for (int b = 0; b < L::kBands; ++b)
                        tma_load_pair(ss + (1 + b) * L::kS, &swmap, 0, (int)(n0 / 128 + b) * tiles + i * L::kTiles, bar);
                }
                __syncwarp();
            }
        }
        // no copy may still be landing when the pair leaves (the first CTA
        // sees both CTAs' copies; they leave together)
        if (rank == 0)
            for (int j = g - S < 0 ? 0 : g - S; j < g; ++j) mbar_wait_bounded(&full[j % S], (uint32_t)(j / S) & 1u);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        // One thread; what it does per stage has to stay below the MMAs' 2 BT cycles.
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = fp4_idesc(FMT, 256, L::kCols);
            const uint32_t base = smem_u32(sm);
            const uint64_t a0 = umma_desc_sw128(base), w0 = umma_desc_sw128(base + L::kABytes);
            const uint64_t s0 = scale_desc(base + L::kABytes + L::kWBytes);
            const int full_stages = (int)(kp / kFp4StageK);  // the last stage may hold 128 k only
            const int total = (SPLIT ? 1 : (units - pair + pairs - 1) / pairs) * (nk - k0);  // stages of this pair's tiles
            bool ok = true;
            int s = 0, slot = 0, g = 0, li = 0;
            uint32_t phase = 0;
            // use `use` of accumulator d waits until the use before has been read
            auto acc_free = [&](int d, int use) {
                if (use > 0 && !tc_wait(&acc_empty[d], (uint32_t)(use - 1) & 1u, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            for (int u = pair; u < units; u += pairs, ++li) {
                // odd tiles of 64 or 192 rows start two columns into their first band of weight scales
                const uint32_t off = BT % 128 == 0 ? 0 : 2 * ((uint32_t)(u / a.tiles_m) & 1);
                const int d = L::kHalves == 2 ? 0 : li & 1;
                if (L::kHalves == 1 && !(ok = acc_free(d, li >> 1))) break;
                for (int i = k0; i < nk; ++i, ++g) {
                    if (!tc_wait(&full[s], phase, abort_flag) ||
                        (L::kSlots < S && g >= L::kSlots &&
                         !tc_wait(&empty[(g - L::kSlots) % S], (uint32_t)((g - L::kSlots) / S) & 1u, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t at = (uint64_t)(s * (L::kStage >> 4));
                    const uint32_t ca = tmem + (uint32_t)(2 * L::kCols + slot * L::kSlotCols), cw = ca + 4 * L::kTiles;
                    const bool whole = i < full_stages;
                    const uint32_t more = i > k0 ? 1u : 0u;
#pragma unroll
                    for (int t = 0; t < L::kTiles; ++t) {
                        if (t < L::kTiles / 2 || whole) {
                            tmem_cp_scales_pair(ca + 4 * t, s0 + at + (uint64_t)(t * kFp4TileBytes >> 4));
#pragma unroll
                            for (int b = 0; b < L::kBands; ++b)
                                tmem_cp_scales_pair(cw + 4 * (t * L::kBands + b),
                                                    s0 + at + (uint64_t)(((1 + b) * L::kS + t * kFp4TileBytes) >> 4));
                        }
                    }
                    auto multiply = [&](int h) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int t = FMT == BITNET_FP4_MX ? j >> 1 : j;
                            const int id = FMT == BITNET_FP4_MX ? (j & 1) * 2 : 0;
                            if (j < 2 || whole)
                                umma_fp4_pair<FMT>(tmem + (uint32_t)((d + h) * L::kCols), a0 + at + 2 * j,
                                                   w0 + at + (uint64_t)(h * (L::kCols / 2 * 128) >> 4) + 2 * j,
                                                   idesc | fp4_scale_id(id), ca + 4 * t,
                                                   cw + 4 * t * L::kBands + off + h * (L::kCols / 32), j > 0 ? 1u : more);
                        }
                    };
                    if (L::kHalves == 2 && i == k0 && !(ok = acc_free(0, li))) break;
                    multiply(0);
                    if constexpr (L::kHalves == 2) {
                        if (i + 1 == nk) umma_commit_pair(&acc_full[0], lead);
                        if (i == k0 && !(ok = acc_free(1, li))) break;
                        multiply(1);
                    }
                    // Only for those who wait: the producers for the stage S further on, this thread for the one kSlots
                    // further on.  (Any other arrival could come after its CTA has left.)
                    if (g + S < total)
                        umma_commit_pair(&empty[s], lead);
                    else if (L::kSlots < S && g + L::kSlots < total)
                        umma_commit_pair(&empty[s], lead, 1u);
                    if (++s == S) s = 0, phase ^= 1;
                    if (++slot == L::kSlots) slot = 0;
                }
                if (!ok) break;
                umma_commit_pair(&acc_full[L::kHalves == 2 ? 1 : d], lead);
            }
            if (!ok) {
                // the MMAs issued so far end before tensor memory is freed (only this CTA waits for them, and the other
                // for this one)
                umma_commit_pair(drain, lead, 1u);
                mbar_wait_bounded(drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- epilogue
        // Two warps share a lane quarter: the first takes the first half of an accumulator's 32-column groups (rounded
        // up), the second the rest.
        constexpr int kGroups = L::kCols / 32, kMost = (kGroups + 1) / 2;
        const int quarter = warp & 3, part = (warp - 2) >> 2;
        const int groups = part == 0 ? kMost : kGroups - kMost;
        const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kMost * 32);
        uint8_t *box = sm + L::kOutAt + (warp - 2) * 4096;
        const float2 gs = fp4_factors(a.ga, a.gw);
        if constexpr (SPLIT) {
            // this pair's sums as they are: rows of BT floats and 16 bytes more, so that the lanes' rows share no banks
            if (warp_wait(&acc_full[0], 0u, abort_flag)) {
                tc_fence_after();
                uint8_t *row = sm + (quarter * 32 + lane) * (BT * 4 + 16) + part * kMost * 128;
#pragma unroll
                for (int c = 0; c < kMost; ++c) {
                    if (c >= groups) break;
                    uint32_t f[32];
                    tmem_ld32(t0 + (uint32_t)(32 * c), f);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(row + c * 128 + 16 * i) =
                            make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                }
            }
        }
        // waits for use `use` of accumulator d, reads this warp's part of it as 16-bit pairs and releases it (where it is
        // used again: any other arrival could come after the first CTA has left)
        auto empty_acc = [&](int d, int use, bool again, uint32_t (&v)[16 * kMost]) -> bool {
            if (!warp_wait(&acc_full[d], (uint32_t)use & 1u, abort_flag)) return false;
            tc_fence_after();
            uint32_t f[32 * kMost];
#pragma unroll
            for (int c = 0; c < kMost; ++c)
                if (c < groups) tmem_ld32(t0 + (uint32_t)(d * L::kCols + 32 * c), f + 32 * c);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (again && lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&acc_empty[d]), lead));
            if (a.ytype == BITNET_FP16)
                pack_all<BITNET_FP16, L::kHalves == 2>(v, f, gs);
            else
                pack_all<BITNET_BF16, L::kHalves == 2>(v, f, gs);
            return true;
        };
        // stores this warp's part: rows of tokens from m0, columns of y from n0
        auto store = [&](int64_t m0, int64_t n0, const uint32_t (&v)[16 * kMost]) {
            const int rows = (int)(a.M - m0 < 32 ? a.M - m0 : 32);
            uint16_t *y = static_cast<uint16_t *>(a.y) + m0 * a.ldy;
#pragma unroll
            for (int c = 0; c < kMost; c += 2) {
                if (c >= groups) break;
                store_box<VEC>(a, box, v, 16 * c, c + 1 < groups ? 8 : 4, y, rows, n0 + 32 * c, lane);
            }
        };
        int li = 0;
        for (int u = pair; !SPLIT && u < units; u += pairs, ++li) {
            const int64_t m0 = (int64_t)(u % a.tiles_m) * 256 + rank * 128 + quarter * 32;
            const int64_t n0 = (int64_t)(u / a.tiles_m) * BT + part * kMost * 32;
            uint32_t v[16 * kMost];
            if constexpr (L::kHalves == 1) {
                if (!empty_acc(li & 1, li >> 1, units - u > 2 * pairs, v)) break;
                store(m0, n0, v);
            } else {
                // both halves are emptied before the first is stored: the next tile waits for them
                uint32_t v1[16 * kMost];
                const bool again = units - u > pairs;
                if (!empty_acc(0, li, again, v) || !empty_acc(1, li, again, v1)) break;
                store(m0, n0, v);
                store(m0, n0 + L::kCols, v1);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    if constexpr (SPLIT) {
        cluster_sync();  // every pair's sums are in its shared memory
        const float2 gs = fp4_factors(a.ga, a.gw);
        const int rows = 128 / a.split, r0 = part_k * rows;
        const int64_t m0 = (int64_t)(pair % a.tiles_m) * 256 + rank * 128, n0 = (int64_t)(pair / a.tiles_m) * BT;
        const bool words = ((reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(2 * a.ldy)) & 7) == 0;
        for (int e = threadIdx.x; e < rows * (BT / 4); e += kFp4PairThreads) {
            const int row = r0 + e / (BT / 4), c = 4 * (e % (BT / 4));
            const int64_t m = m0 + row, n = n0 + c;
            if (m >= a.M || n >= a.N) continue;
            const uint32_t at = smem_u32(sm) + (uint32_t)(row * (BT * 4 + 16) + c * 4);
            float4 t = ld_cluster_v4(map_rank(at, rank));
            for (int q = 1; q < a.split; ++q) {
                const float4 o = ld_cluster_v4(map_rank(at, 2 * q + rank));
                t.x += o.x, t.y += o.y, t.z += o.z, t.w += o.w;
            }
            const float v[4] = {fp4_scaled(t.x, gs), fp4_scaled(t.y, gs), fp4_scaled(t.z, gs), fp4_scaled(t.w, gs)};
            if (words && n + 4 <= a.N) {
                const uint2 p = a.ytype == BITNET_FP16
                                    ? make_uint2(pack2<BITNET_FP16>(v[0], v[1]), pack2<BITNET_FP16>(v[2], v[3]))
                                    : make_uint2(pack2<BITNET_BF16>(v[0], v[1]), pack2<BITNET_BF16>(v[2], v[3]));
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + m * a.ldy + n) = p;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.N) fp4_store(a.y, m * a.ldy + n + i, v[i], a.ytype);
            }
        }
    }
    __syncthreads();
    cluster_sync_relaxed();  // neither CTA signals the other or reads its shared memory any more
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmem) : "memory");
    }
}

}  // namespace bitnet

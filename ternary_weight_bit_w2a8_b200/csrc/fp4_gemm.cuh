// fp4_gemm.cuh -- product of two microscaled 4-bit matrices on the
// 5th-generation tensor cores (tcgen05.mma with block scales, fp32
// accumulators in tensor memory).
//
//   y[m, n] = ga * gw * sum_k (a[m, k] sa[m, k / B]) (w[n, k] sw[n, k / B])
//
// The tensor core multiplies e2m1 elements and their block scales itself: code
// rows go to shared memory as they are stored (K-major, two elements a byte,
// 256 k = 128 bytes to a swizzled row) and scale tiles (128 rows x 4 blocks,
// 512 bytes) from there to tensor memory, 32 lanes x 4 columns repeated over
// the four lane quarters, which is the order the tiles are stored in.
#pragma once

#include "fp4.cuh"
#include "gemm_tc.cuh"

namespace bitnet {

constexpr int kFp4Rows = 128;     // rows of the P operand per tile (UMMA M)
constexpr int kFp4StageK = 256;   // k per stage: a 128-byte swizzled row of codes
constexpr int kFp4Threads = 192;  // producer, MMA issuer, 4 epilogue (and quantiser) warps
constexpr int kFp4MaxSplit = 8;   // largest portable cluster
constexpr int kFp4FusedTokens = 16;

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// One lane of a converged warp, always the same one.  The loops that issue
// MMAs and copies run on the whole warp and issue under this: with `lane == 0`
// in its place the compiler cannot see that one thread issues, and a 256-k
// stage of the pair kernel below took 727 cycles instead of its 512.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Whole-warp bounded wait: every lane gives up or none does.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag)) != 0;
}

// Instruction descriptor: e2m1 x e2m1, fp32 accumulate, K-major, M = m, N = n,
// scale type 1 (e8m0) or 0 (e4m3); the two scale ids (which byte of a column
// holds the first scale) are added per instruction.
__host__ __device__ constexpr uint32_t fp4_idesc(int fmt, int m, int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((fmt == BITNET_FP4_MX ? 1u : 0u) << 23) |
           ((uint32_t)(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t fp4_scale_id(int id) { return ((uint32_t)id << 4) | ((uint32_t)id << 29); }

// D (+)= (A scaled) x (B scaled): 64 k.
template <int FMT>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
    if (FMT == BITNET_FP4_MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// Descriptor of a scale tile in shared memory (512 bytes, 16-byte aligned),
// unswizzled: 8-row groups of 16-byte rows, 128 bytes from group to group.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// One scale tile to four tensor-memory columns, repeated over the four lane
// quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void fp4_store(void *y, int64_t i, float v, int dtype) {
    if (dtype == BITNET_FP16)
        static_cast<__half *>(y)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ few tokens
// Up to 128 tokens: reading the weights bounds the call.  The weights are the
// MMA's row operand (128 rows of them a tile), the tokens its BT columns, so
// that one pass over the weights serves all tokens.  Tiles are few (20 for
// 2560 rows), so a cluster of up to 8 CTAs shares a tile, each with a range of
// k; the CTAs add their fp32 sums up through distributed shared memory, in
// rank order, each for its share of the rows.  No workspace, no atomics, and
// the same bits every time.  Two CTAs fit an SM, so that one's start and end
// overlap the other's loads.
//   Before the launch-chain wait the first boxes of the weights are only asked
// into L2: what an earlier kernel still writes is read after the wait.
//   QX: up to 16 tokens of x are quantised by the epilogue warps stage by
// stage, straight into the swizzled operand rows and scale tiles, with the
// arithmetic of fp4_quant_kernel.
struct Fp4SmallArgs {
    const uint8_t *sw, *sa;  // scale tiles of the weights and of the tokens
    const void *x;           // QX: the tokens [M, K], row stride ldx
    int64_t ldx;
    int xtype, ytype;
    int M;
    int64_t N, K, ldy;
    const float *ga, *gw;
    void *y;
    int split;               // CTAs per cluster
};

template <int FMT, int BT>
struct Fp4Small {
    static constexpr int kTiles = FMT == BITNET_FP4_MX ? 2 : 4;  // scale tiles per stage and 128 rows
    static constexpr int kPBytes = kFp4Rows * 128, kQBytes = BT * 128, kS = kTiles * kFp4TileBytes;
    static constexpr int kStage = kPBytes + kQBytes + 2 * kS;
    static constexpr int kStages = 110 * 1024 / kStage < 6 ? 110 * 1024 / kStage : 6;
    static constexpr int kBars = kStages * kStage;
    static constexpr int kBytes = kBars + (2 * kStages + 2) * 8 + 16;
    static constexpr int kSlotCols = 8 * kTiles;                 // tensor-memory columns of a stage's scales
    static constexpr int kNeed = BT + 2 * kSlotCols;
    static constexpr int kCols = kNeed <= 32 ? 32 : kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : 256;
    static_assert(kNeed <= 256 && kStages >= 3 && BT % 16 == 0 && BT <= 128, "tile");
    static_assert(kStage % 1024 == 0 && kQBytes % 1024 == 0, "swizzled rows");
    static_assert(kFp4Rows * BT * 4 <= kBars, "partial sums take the stages' place");
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// 8 values of row m from column k for the quantiser warps.
__device__ __forceinline__ void fp4_load8_any(const Fp4SmallArgs &a, int m, int64_t k, float (&v)[8]) {
    if (a.xtype == BITNET_FP32) {
        const float *r = static_cast<const float *>(a.x) + m * a.ldx;
        fp4_load8<BITNET_FP32>(r, k, a.K, (reinterpret_cast<uintptr_t>(r) & 15) == 0, v);
    } else if (a.xtype == BITNET_FP16) {
        const __half *r = static_cast<const __half *>(a.x) + m * a.ldx;
        fp4_load8<BITNET_FP16>(r, k, a.K, (reinterpret_cast<uintptr_t>(r) & 15) == 0, v);
    } else {
        const __nv_bfloat16 *r = static_cast<const __nv_bfloat16 *>(a.x) + m * a.ldx;
        fp4_load8<BITNET_BF16>(r, k, a.K, (reinterpret_cast<uintptr_t>(r) & 15) == 0, v);
    }
}

template <int FMT, int BT, bool QX>
__global__ void __launch_bounds__(kFp4Threads, 2)
    fp4_small_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                     const Fp4SmallArgs a) {
    using L = Fp4Small<FMT, BT>;
    static_assert(!QX || BT >= kFp4FusedTokens, "fused tokens");
    constexpr int S = L::kStages;
    constexpr int B = FMT == BITNET_FP4_MX ? 32 : 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::kBars);
    uint64_t *empty = full + S;
    uint64_t *done = empty + S;
    uint64_t *drain = done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)a.split), tile = (int)(blockIdx.x / (unsigned)a.split);
    const int64_t kp = k_pad(a.K);
    const int nk = (int)ceil_div(kp, kFp4StageK);
    // this CTA's stages (split <= nk, so there is one at least)
    const int i0 = (int)((int64_t)nk * rank / a.split), n_i = (int)((int64_t)nk * (rank + 1) / a.split) - i0;
    const int64_t tiles = fp4_scale_tiles(a.K, FMT);
    const uint8_t *sw = a.sw + (int64_t)tile * tiles * kFp4TileBytes;
    auto scale_bytes = [&](int i) {  // of stage i: the last one may have fewer tiles
        const int64_t left = tiles - (int64_t)i * L::kTiles;
        return (uint32_t)(left < L::kTiles ? left : L::kTiles) * kFp4TileBytes;
    };

    if (threadIdx.x == 0) {
        prefetch_tensormap(&wmap);
        if (!QX) prefetch_tensormap(&amap);
        for (int i = 0; i < n_i && i < S; ++i) {
            tma_prefetch_2d(&wmap, (i0 + i) * 128, tile * kFp4Rows);
            prefetch_l2_bulk(sw + (int64_t)(i0 + i) * L::kS, scale_bytes(i0 + i));
        }
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], QX ? 5 : 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(L::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (QX) {  // token rows and scales that no token fills: zero in every stage
        constexpr int kWords = (L::kQBytes + L::kS) / 16;
        for (int i = threadIdx.x; i < S * kWords; i += kFp4Threads) {
            const int s = i / kWords, o = (i % kWords) * 16;
            *reinterpret_cast<uint4 *>(sm + s * L::kStage + L::kPBytes + (o < L::kQBytes ? o : o + L::kS)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        int i = 0;
        for (; i < n_i; ++i) {
            const int s = i % S, gi = i0 + i;
            if (i >= S && !warp_wait(&empty[s], (uint32_t)(i / S - 1) & 1u, abort_flag)) break;
            if (elect_one()) {
                uint8_t *st = sm + s * L::kStage;
                const uint32_t sb = scale_bytes(gi);
                mbar_arrive_expect_tx(&full[s], QX ? L::kPBytes + sb : L::kPBytes + L::kQBytes + 2 * sb);
                tma_load_2d(st, &wmap, gi * 128, tile * kFp4Rows, &full[s]);
                uint8_t *ss = st + L::kPBytes + L::kQBytes;
                bulk_load(ss, sw + (int64_t)gi * L::kS, sb, &full[s]);
                if (!QX) {
                    tma_load_2d(st + L::kPBytes, &amap, gi * 128, 0, &full[s]);
                    bulk_load(ss + L::kS, a.sa + (int64_t)gi * L::kS, sb, &full[s]);
                }
            }
            __syncwarp();
        }
        // no copy may still be landing when the CTA leaves (QX: a stage's
        // barrier also waits for the quantisers, which stop on an abort; the
        // wait is bounded)
        for (int j = i - S < 0 ? 0 : i - S; j < i; ++j) mbar_wait_bounded(&full[j % S], (uint32_t)(j / S) & 1u);
    } else if (warp == 1) {
        constexpr uint32_t idesc = fp4_idesc(FMT, kFp4Rows, BT);
        bool ok = true;
        for (int i = 0; i < n_i; ++i) {
            const int s = i % S;
            // two sets of scale columns take turns: the MMAs that read this
            // one, two stages ago, are done
            ok = warp_wait(&full[s], (uint32_t)(i / S) & 1u, abort_flag) &&
                 (i < 2 || warp_wait(&empty[(i - 2) % S], (uint32_t)((i - 2) / S) & 1u, abort_flag));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t pa = smem_u32(sm + s * L::kStage), qa = pa + L::kPBytes;
                const uint32_t spa = qa + L::kQBytes, sqa = spa + L::kS;
                const uint32_t cp = tmem + (uint32_t)(BT + (i & 1) * L::kSlotCols), cq = cp + 4 * L::kTiles;
                const int64_t left = (kp - (int64_t)(i0 + i) * kFp4StageK) / 64;
                const int steps = (int)(left < 4 ? left : 4);
#pragma unroll
                for (int t = 0; t < L::kTiles; ++t) {
                    tmem_cp_scales(cp + 4 * t, scale_desc(spa + t * kFp4TileBytes));
                    tmem_cp_scales(cq + 4 * t, scale_desc(sqa + t * kFp4TileBytes));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < steps) {
                        const int t = FMT == BITNET_FP4_MX ? j >> 1 : j;
                        const int id = FMT == BITNET_FP4_MX ? (j & 1) * 2 : 0;
                        umma_fp4<FMT>(tmem, umma_desc_sw128(pa + 32 * j), umma_desc_sw128(qa + 32 * j),
                                      idesc | fp4_scale_id(id), cp + 4 * t, cq + 4 * t, (i > 0 || j > 0) ? 1u : 0u);
                    }
                }
                umma_commit(&empty[s]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(ok ? done : drain);
        __syncwarp();
        // on an abort the MMAs issued so far end before tensor memory is freed
        if (!ok) mbar_wait_bounded(drain, 0);
    } else {
        if (QX) {
            // warp w of four takes tokens w, w + 4, ...; a lane 8 of a stage's 256 k.  The next stage's values are
            // on their way while this one's are quantised.
            const int w = warp - 2;
            constexpr int R = kFp4FusedTokens / 4;
            const float inv = a.ga != nullptr ? __frcp_rn(*a.ga) : 1.0f;
            float z[R][8];
            auto load = [&](int i) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (w + 4 * r < a.M) fp4_load8_any(a, w + 4 * r, (int64_t)(i0 + i) * kFp4StageK + 8 * lane, z[r]);
            };
            load(0);
            for (int i = 0; i < n_i; ++i) {
                const int s = i % S;
                // the lanes stop together (they shuffle below)
                if (i >= S && !warp_wait(&empty[s], (uint32_t)(i / S - 1) & 1u, abort_flag)) break;
                uint8_t *q = sm + s * L::kStage + L::kPBytes, *sq = q + L::kQBytes + L::kS;
                float v[R][8];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[r][e] = z[r][e];
                if (i + 1 < n_i) load(i + 1);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int m = w + 4 * r;
                    if (m < a.M) {
                        uint32_t top = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            v[r][e] = __fmul_rn(v[r][e], inv);
                            const uint32_t b = __float_as_uint(v[r][e]) & 0x7fffffffu;
                            top = b > top ? b : top;
                        }
#pragma unroll
                        for (int o = 1; o < B / 8; o *= 2) {
                            const uint32_t t = __shfl_xor_sync(0xffffffffu, top, o);
                            top = t > top ? t : top;
                        }
                        const Fp4Scale sc = fp4_scale<FMT>(top);
                        // 16-byte chunk c of row m lies at chunk c ^ (m % 8)
                        *reinterpret_cast<uint32_t *>(q + m * 128 + ((((lane >> 2) ^ m) & 7) << 4) + 4 * (lane & 3)) =
                            fp4_codes8<FMT>(v[r], sc, top < 0x7f800000u);
                        if (lane % (B / 8) == 0)
                            sq[(lane * 8 / (4 * B)) * kFp4TileBytes + 16 * m + ((lane * 8 / B) & 3)] = (uint8_t)sc.byte;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
            __syncwarp();
        }
        const int quarter = warp & 3;
        const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16);
        const int row = quarter * 32 + lane;
        if (warp_wait(done, 0u, abort_flag)) {
            tc_fence_after();
            const float g = (a.ga != nullptr ? *a.ga : 1.0f) * (a.gw != nullptr ? *a.gw : 1.0f);
            const int64_t n = (int64_t)tile * kFp4Rows + row;
            float *part = reinterpret_cast<float *>(sm);
#pragma unroll 1
            for (int c = 0; c < BT && c < a.M; c += 16) {
                uint32_t v[16];
                tmem_ld16(t0 + (uint32_t)c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (c + i >= a.M) break;
                    if (a.split > 1)
                        part[(c + i) * kFp4Rows + row] = __uint_as_float(v[i]);
                    else if (n < a.N)
                        fp4_store(a.y, (c + i) * a.ldy + n, __fmul_rn(__uint_as_float(v[i]), g), a.ytype);
                }
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    if (a.split > 1) {
        cluster_sync();  // every CTA's sums are in its shared memory
        const float g = (a.ga != nullptr ? *a.ga : 1.0f) * (a.gw != nullptr ? *a.gw : 1.0f);
        const int rows = kFp4Rows / a.split, r0 = rank * rows;
        const uint32_t base = smem_u32(sm);
        for (int e = threadIdx.x; e < a.M * rows; e += kFp4Threads) {
            const int c = e / rows, row = r0 + e % rows;
            const int64_t n = (int64_t)tile * kFp4Rows + row;
            const uint32_t at = base + (uint32_t)(c * kFp4Rows + row) * 4;
            float v[kFp4MaxSplit];
#pragma unroll
            for (int r = 0; r < kFp4MaxSplit; ++r) v[r] = r < a.split ? ld_cluster(map_rank(at, (uint32_t)r)) : 0.0f;
            float sum = v[0];
#pragma unroll
            for (int r = 1; r < kFp4MaxSplit; ++r) sum += v[r];
            if (n < a.N) fp4_store(a.y, c * a.ldy + n, __fmul_rn(sum, g), a.ytype);
        }
        cluster_sync();  // nobody reads this CTA's shared memory any more
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
}

}  // namespace bitnet

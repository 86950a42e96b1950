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
constexpr int kFp4Threads = 192;  // producer, MMA issuer, 4 epilogue warps

struct Fp4GemmArgs {
    const uint8_t *sp, *sq;   // scale tiles of the P and Q operands
    int64_t P, Q;             // their rows
    int64_t K;
    int64_t stride_p, stride_q;  // y strides: element (p, q) is y[p * stride_p + q * stride_q]
    const float *ga, *gw;     // tensor scales or null
    void *y;
    int tiles_p;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
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

// One scale tile from shared memory (512 bytes, 16-byte aligned) to four
// tensor-memory columns, repeated over the four lane quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr) {
    // unswizzled: 8-row groups of 16-byte rows, 128 bytes from group to group
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int FMT, int BT>
struct Fp4Smem {
    static constexpr int kTiles = FMT == BITNET_FP4_MX ? 2 : 4;     // scale tiles per stage and 128 rows
    static constexpr int kQTiles = (BT + 127) / 128;
    static constexpr int kPBytes = kFp4Rows * 128, kQBytes = BT * 128;
    static constexpr int kSP = kTiles * kFp4TileBytes, kSQ = kQTiles * kTiles * kFp4TileBytes;
    static constexpr int kStage = kPBytes + kQBytes + kSP + kSQ;
    static constexpr int kStages = 196 * 1024 / kStage < 8 ? 196 * 1024 / kStage : 8;
    static constexpr int kBars = kStages * kStage;
    static constexpr int kBytes = kBars + (2 * kStages + 2) * 8 + 16;
    static constexpr int kSlotCols = 4 * kTiles * (1 + kQTiles);    // tensor-memory columns of a stage's scales
    static constexpr int kNeed = BT + 2 * kSlotCols;
    static constexpr int kCols = kNeed <= 32 ? 32 : kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static_assert(kNeed <= 512 && kStages >= 3 && BT % 8 == 0, "tile");
    static_assert(kStage % 1024 == 0 && kPBytes % 1024 == 0 && kQBytes % 1024 == 0, "swizzled rows");
};

// One CTA per tile of 128 P rows x BT Q rows.
template <int FMT, int BT, int DT>
__global__ void __launch_bounds__(kFp4Threads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap qmap,
                    const Fp4GemmArgs a) {
    using L = Fp4Smem<FMT, BT>;
    using T = typename Fp4Type<DT>::T;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::kBars);
    uint64_t *empty = full + S;
    uint64_t *done = empty + S;
    uint64_t *drain = done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tp = blockIdx.x % a.tiles_p, tq = blockIdx.x / a.tiles_p;
    const int64_t p0 = (int64_t)tp * kFp4Rows, q0 = (int64_t)tq * BT;
    const int64_t kp = k_pad(a.K);
    const int nk = (int)ceil_div(kp, kFp4StageK);

    if (threadIdx.x == 0) {
        prefetch_tensormap(&pmap);
        prefetch_tensormap(&qmap);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            const int64_t tiles = fp4_scale_tiles(a.K, FMT);
            const int64_t qbands = ceil_div(a.Q, kFp4TileRows);
            int i = 0;
            for (; i < nk; ++i) {
                const int s = i % S;
                if (i >= S && !tc_wait(&empty[s], (uint32_t)(i / S - 1) & 1u, abort_flag)) break;
                uint8_t *st = sm + s * L::kStage;
                const int64_t t0 = (int64_t)i * L::kTiles;
                const uint32_t sb = (uint32_t)(tiles - t0 < L::kTiles ? tiles - t0 : L::kTiles) * kFp4TileBytes;
                const int nq = (int)(qbands - q0 / 128 < L::kQTiles ? qbands - q0 / 128 : L::kQTiles);
                mbar_arrive_expect_tx(&full[s], L::kPBytes + L::kQBytes + sb * (1 + nq));
                tma_load_2d(st, &pmap, i * 128, (int)p0, &full[s]);
                tma_load_2d(st + L::kPBytes, &qmap, i * 128, (int)q0, &full[s]);
                uint8_t *ss = st + L::kPBytes + L::kQBytes;
                bulk_load(ss, a.sp + ((int64_t)tp * tiles + t0) * kFp4TileBytes, sb, &full[s]);
                for (int q = 0; q < nq; ++q)
                    bulk_load(ss + L::kSP + q * L::kSP, a.sq + ((q0 / 128 + q) * tiles + t0) * kFp4TileBytes, sb,
                              &full[s]);
            }
            // no copy may still be landing when the CTA leaves
            for (int j = i - S < 0 ? 0 : i - S; j < i; ++j) mbar_wait_bounded(&full[j % S], (uint32_t)(j / S) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = fp4_idesc(FMT, kFp4Rows, BT);
            bool ok = true;
            for (int i = 0; i < nk; ++i) {
                const int s = i % S;
                // two sets of scale columns take turns: the MMAs that read this
                // one, two stages ago, are done
                if (!tc_wait(&full[s], (uint32_t)(i / S) & 1u, abort_flag) ||
                    (i >= 2 && !tc_wait(&empty[(i - 2) % S], (uint32_t)((i - 2) / S) & 1u, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t pa = smem_u32(sm + s * L::kStage), qa = pa + L::kPBytes;
                const uint32_t spa = qa + L::kQBytes, sqa = spa + L::kSP;
                const uint32_t cp = tmem + (uint32_t)(BT + (i & 1) * L::kSlotCols), cq = cp + 4 * L::kTiles;
                const int steps = (int)((kp - (int64_t)i * kFp4StageK) / 64 < 4 ? (kp - (int64_t)i * kFp4StageK) / 64 : 4);
#pragma unroll
                for (int t = 0; t < L::kTiles; ++t) {
                    tmem_cp_scales(cp + 4 * t, spa + t * kFp4TileBytes);
#pragma unroll
                    for (int q = 0; q < L::kQTiles; ++q)
                        tmem_cp_scales(cq + 4 * (t * L::kQTiles + q), sqa + q * L::kSP + t * kFp4TileBytes);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < steps) {
                        const int t = FMT == BITNET_FP4_MX ? j >> 1 : j;
                        const int id = FMT == BITNET_FP4_MX ? (j & 1) * 2 : 0;
                        umma_fp4<FMT>(tmem, umma_desc_sw128(pa + 32 * j), umma_desc_sw128(qa + 32 * j),
                                      idesc | fp4_scale_id(id), cp + 4 * t, cq + 4 * t * L::kQTiles,
                                      (i > 0 || j > 0) ? 1u : 0u);
                    }
                }
                umma_commit(&empty[s]);
            }
            if (ok) {
                umma_commit(done);
            } else {
                umma_commit(drain);  // the MMAs issued so far end before tensor memory is freed
                mbar_wait_bounded(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;
        const uint32_t tq_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        if (tc_wait(done, 0u, abort_flag)) {
            tc_fence_after();
            const float g = (a.ga != nullptr ? *a.ga : 1.0f) * (a.gw != nullptr ? *a.gw : 1.0f);
            const int64_t p = p0 + quarter * 32 + lane;
            T *y = static_cast<T *>(a.y);
            constexpr int kLd = BT < 16 ? BT : 16;
#pragma unroll 1
            for (int c = 0; c < BT; c += kLd) {
                uint32_t v[16];
                tmem_ld16(tq_addr + (uint32_t)c, v);
#pragma unroll
                for (int i = 0; i < kLd; ++i)
                    if (p < a.P && q0 + c + i < a.Q)
                        y[p * a.stride_p + (q0 + c + i) * a.stride_q] = Fp4Type<DT>::from_f(__fmul_rn(__uint_as_float(v[i]), g));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
}

}  // namespace bitnet

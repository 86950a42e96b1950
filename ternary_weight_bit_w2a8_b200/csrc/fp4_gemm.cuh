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

constexpr int kFp4Threads = 192;  // producer, MMA issuer, 4 epilogue (and quantiser) warps
// Tokens that are quantised inside the product's launch; callers count on needing
// no workspace up to there.  In a graph, one launch against quantising first: 1
// token 4.9 to 6.7 us and 6.1 to 7.7 for 2560 x 6912 to 13824 x 2560, 16 tokens
// 6.7 to 8.2 and 6.7 to 8.8.  But every CTA quantises all tokens of its range of
// k: with 27648 rows and more one token takes as long either way, and 4 to 16
// take longer (55296 x 5120 MX: 28.6 to 33.4 us, quantised first 25.8 to 26.5).
constexpr int kFp4FusedTokens = 16;
constexpr int kFp4Prefetch = 4;  // stages of weights asked into L2 before the launch-chain wait

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

// ga * gw in two factors, by which a sum is multiplied one after the other:
// their product and 1, or, where fp32 does not hold that as a normal number
// (tensors of values around 1e-20 have such scales, and sums of 1e8 beside
// them), 2^126 times the product and 2^-126, or 2^-126 times it and 2^126.  The
// power goes to the smaller scale first, exactly: below 2^-63 in the one case,
// above 1 in the other.
__device__ __forceinline__ float2 fp4_factors(const float *ga, const float *gw) {
    const float a = ga != nullptr ? *ga : 1.0f, b = gw != nullptr ? *gw : 1.0f, p = fabsf(__fmul_rn(a, b));
    const bool below = p < 0x1p-126f, above = p == __uint_as_float(0x7f800000u), swap = fabsf(a) > fabsf(b);
    const float up = below ? 0x1p126f : (above ? 0x1p-126f : 1.0f), down = below ? 0x1p-126f : (above ? 0x1p126f : 1.0f);
    return make_float2(__fmul_rn(__fmul_rn(swap ? b : a, up), swap ? a : b), down);
}
__device__ __forceinline__ float fp4_scaled(float sum, float2 g) { return __fmul_rn(__fmul_rn(sum, g.x), g.y); }

// ------------------------------------------------------------------ few tokens
// Up to 64 tokens: reading the weights bounds the call.  The weights are the
// MMA's row operand (128 rows of them a tile), the tokens its BT columns, so
// that one pass over the weights serves all tokens.  Tiles are few (20 for
// 2560 rows), so a cluster of up to 8 CTAs shares a tile, each with a range of
// k; the CTAs add their fp32 sums up through distributed shared memory, in
// rank order, each for its share of the rows.  No workspace, no atomics, and
// the same bits every time.  Three CTAs fit an SM (two from 17 tokens up), so
// that one's start and end overlap the others' loads.
//   Launch chain: before the wait for the kernel before, the first weights are
// only asked into L2 (what that kernel still writes is read after the wait).
// The next kernel may start once this one has asked for its last weights: its
// CTAs then find room and warm L2 while this one multiplies, exchanges and
// stores (1 x 13824 x 5120 MX 8.9 -> 8.0 us); started with this one's first
// loads they took its bandwidth instead (9.2 us).
//   QX: up to 16 tokens of x are quantised by the epilogue warps stage by
// stage, straight into the swizzled operand rows and scale tiles, with the
// arithmetic of fp4_quant_kernel.
struct Fp4SmallArgs {
    const uint8_t *sw, *sa;  // scale tiles of the weights and of the tokens
    const void *x;           // QX: the tokens [M, K], row stride ldx
    int64_t ldx;
    int ytype;
    int M;
    int64_t N, K, ldy;
    const float *ga, *gw;
    void *y;
    int split;               // CTAs per cluster
    int test_stall;          // the first CTA never asks for its first stage (test of the bounded waits)
};

template <int FMT, int BT>
struct Fp4Small {
    static constexpr int kTiles = FMT == BITNET_FP4_MX ? 2 : 4;  // scale tiles per stage and 128 rows
    static constexpr int kPBytes = kFp4Rows * 128, kQBytes = BT * 128, kS = kTiles * kFp4TileBytes;
    static constexpr int kStage = kPBytes + kQBytes + 2 * kS;
    static constexpr int kCtas = BT <= 16 ? 3 : 2;               // CTAs per SM
    static constexpr int kStages = (kCtas == 3 ? 73 : 111) * 1024 / kStage;
    static constexpr int kBars = kStages * kStage;
    static constexpr int kBytes = kBars + (2 * kStages + 2) * 8 + 16;
    static constexpr int kSlotCols = 8 * kTiles;                 // tensor-memory columns of a stage's scales
    static constexpr int kNeed = BT + kStages * kSlotCols;
    static constexpr int kCols = kNeed <= 32 ? 32 : kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : 256;
    static_assert(kNeed <= 256 && kCtas * kCols <= 512 && kStages >= 3 && BT % 16 == 0 && BT <= 64, "tile");
    static_assert(kStage % 1024 == 0 && kQBytes % 1024 == 0, "swizzled rows");
    static_assert(kFp4Rows * BT * 4 <= kBars, "partial sums take the stages' place");
    static_assert(BT >= 16, "accumulators are read 16 columns at a time");
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

constexpr int kFp4Quantised = -1;  // XT: the tokens come quantised

// The quantiser warps of the small kernel: warp w of four.  As in
// fp4_quant_kernel a lane takes 32 bytes of a token; so a warp takes two tokens
// at a time (one of fp32), and its tokens of a stage are w RW, w RW + 1, ...,
// then 4 RW further.  The next stage's values are on their way while this one's
// are quantised.
template <int FMT, int BT, int XT>
__device__ __forceinline__ void fp4_quantise_stages(const Fp4SmallArgs &a, uint8_t *sm, uint64_t *full, uint64_t *empty,
                                                    int i0, int n_i, int w, int warp_lane, volatile int *abort_flag) {
    using L = Fp4Small<FMT, BT>;
    using T = typename Fp4Type<XT>::T;
    constexpr int S = L::kStages, B = FMT == BITNET_FP4_MX ? 32 : 16;
    constexpr int V = Fp4Raw<XT>::kValues, kLanes = kFp4StageK / V, RW = 32 / kLanes;
    constexpr int kTurns = kFp4FusedTokens / (4 * RW);
    const int lane = warp_lane % kLanes, m0 = w * RW + warp_lane / kLanes;
    const T *x = static_cast<const T *>(a.x);
    const uintptr_t where = reinterpret_cast<uintptr_t>(x) | (uintptr_t)(a.ldx * (int64_t)sizeof(T));
    const float inv = a.ga != nullptr ? __frcp_rn(*a.ga) : 1.0f;
    Fp4Raw<XT> next[kTurns];
    auto load = [&](int i) {
        const int64_t k = (int64_t)(i0 + i) * kFp4StageK + V * lane;
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int m = m0 + 4 * RW * t;
            if (m >= a.M) continue;
            if ((where & 15) == 0) {
                next[t] = fp4_load32<XT>(x + m * a.ldx, k, a.K, (where & 31) == 0);
            } else {
                alignas(16) T v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = k + e < a.K ? x[m * a.ldx + k + e] : T(0.0f);
#pragma unroll
                for (int e = 0; e < 8; ++e) next[t].w[e] = reinterpret_cast<const uint32_t *>(v)[e];
            }
        }
    };
    load(0);
    int s = 0;
    uint32_t phase = 1;  // of `empty`: passes at once in the first round
    for (int i = 0; i < n_i; ++i) {
        // the lanes stop together (they shuffle below)
        if (!warp_wait(&empty[s], phase, abort_flag)) break;
        uint8_t *q = sm + s * L::kStage + L::kPBytes, *sq = q + L::kQBytes + L::kS;
        Fp4Raw<XT> v[kTurns];
#pragma unroll
        for (int t = 0; t < kTurns; ++t) v[t] = next[t];
        if (i + 1 < n_i) load(i + 1);
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int m = m0 + 4 * RW * t;
            if (m - warp_lane / kLanes >= a.M) break;  // (both tokens of the warp)
            uint32_t top = m < a.M ? fp4_absmax<XT>(v[t]) : 0u;
            top = __float_as_uint(__fmul_rn(__uint_as_float(top), inv)) & 0x7fffffffu;
#pragma unroll
            for (int o = 1; o < B / V; o *= 2) {
                const uint32_t u = __shfl_xor_sync(0xffffffffu, top, o);
                top = u > top ? u : top;
            }
            if (m >= a.M) continue;
            const Fp4Scale sc = fp4_scale<FMT>(top);
            uint32_t c[V / 8];
#pragma unroll
            for (int h = 0; h < V / 8; ++h) {
                uint64_t p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = fp4_pair<XT>(v[t], 4 * h + e);
                c[h] = fp4_codes8<FMT>(p, inv, sc, top < 0x7f800000u);
            }
            // 16-byte piece p of token m lies at piece p ^ (m % 8) of its row
            const int byte = V / 2 * lane;
            uint8_t *to = q + m * 128 + ((((byte >> 4) ^ m) & 7) << 4) + (byte & 15);
            if constexpr (V == 16)
                *reinterpret_cast<uint2 *>(to) = make_uint2(c[0], c[1]);
            else
                *reinterpret_cast<uint32_t *>(to) = c[0];
            if (lane % (B / V) == 0) sq[(lane * V / (4 * B)) * kFp4TileBytes + 16 * m + (lane * V / B & 3)] = (uint8_t)sc.byte;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (warp_lane == 0) mbar_arrive(&full[s]);
        if (++s == S) s = 0, phase ^= 1;
    }
    __syncwarp();
}

template <int FMT, int BT, int XT>
__global__ void __launch_bounds__(kFp4Threads, Fp4Small<FMT, BT>::kCtas)
    fp4_small_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                     const Fp4SmallArgs a) {
    using L = Fp4Small<FMT, BT>;
    constexpr bool QX = XT != kFp4Quantised;
    static_assert(!QX || BT >= kFp4FusedTokens, "fused tokens");
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
        for (int i = 0; i < n_i && i < kFp4Prefetch; ++i) {
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

    if (warp == 0) {
        if (n_i <= S) pdl_launch_dependents();
        int i = 0;
        for (; i < n_i; ++i) {
            const int s = i % S, gi = i0 + i;
            if (i >= S && !warp_wait(&empty[s], (uint32_t)(i / S - 1) & 1u, abort_flag)) break;
            if (a.test_stall && blockIdx.x == 0 && i == 0) continue;
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
        if (n_i > S) pdl_launch_dependents();
        // no copy may still be landing when the CTA leaves (QX: a stage's
        // barrier also waits for the quantisers, which stop on an abort; the
        // wait is bounded)
        for (int j = i - S < 0 ? 0 : i - S; j < i; ++j) mbar_wait_bounded(&full[j % S], (uint32_t)(j / S) & 1u);
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = fp4_idesc(FMT, kFp4Rows, BT);
            const uint32_t base = smem_u32(sm);
            const uint64_t w0 = umma_desc_sw128(base), a0 = umma_desc_sw128(base + L::kPBytes);
            const uint64_t s0 = scale_desc(base + L::kPBytes + L::kQBytes);
            const int full_stages = (int)(kp / kFp4StageK) - i0;  // the last stage may hold 128 k only
            bool ok = true;
            int s = 0;
            uint32_t phase = 0;
            for (int i = 0; i < n_i; ++i) {
                if (!tc_wait(&full[s], phase, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t at = (uint64_t)(s * (L::kStage >> 4));
                const uint32_t cw = tmem + (uint32_t)(BT + s * L::kSlotCols), ca = cw + 4 * L::kTiles;
                const bool whole = i < full_stages;
#pragma unroll
                for (int t = 0; t < L::kTiles; ++t) {
                    if (t < L::kTiles / 2 || whole) {
                        tmem_cp_scales(cw + 4 * t, s0 + at + (uint64_t)(t * kFp4TileBytes >> 4));
                        tmem_cp_scales(ca + 4 * t, s0 + at + (uint64_t)((L::kS + t * kFp4TileBytes) >> 4));
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = FMT == BITNET_FP4_MX ? j >> 1 : j;
                    const int id = FMT == BITNET_FP4_MX ? (j & 1) * 2 : 0;
                    if (j < 2 || whole)
                        umma_fp4<FMT>(tmem, w0 + at + 2 * j, a0 + at + 2 * j, idesc | fp4_scale_id(id), cw + 4 * t,
                                      ca + 4 * t, j > 0 ? 1u : (uint32_t)(i > 0));
                }
                // (an arrival that no load waits for could come after the CTA has left)
                if (i + S < n_i) umma_commit(&empty[s]);
                if (++s == S) s = 0, phase ^= 1;
            }
            umma_commit(ok ? done : drain);
            // on an abort the MMAs issued so far end before tensor memory is freed
            if (!ok) mbar_wait_bounded(drain, 0);
        }
        __syncwarp();
    } else {
        if constexpr (QX) fp4_quantise_stages<FMT, BT, XT>(a, sm, full, empty, i0, n_i, warp - 2, lane, abort_flag);
        const int quarter = warp & 3;
        const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16);
        const int row = quarter * 32 + lane;
        const float2 g = fp4_factors(a.ga, a.gw);
        if (warp_wait(done, 0u, abort_flag)) {
            tc_fence_after();
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
                        fp4_store(a.y, (c + i) * a.ldy + n, fp4_scaled(__uint_as_float(v[i]), g), a.ytype);
                }
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    if (a.split > 1) {
        cluster_sync();  // every CTA's sums are in its shared memory
        const float2 g = fp4_factors(a.ga, a.gw);
        // four neighbouring rows of a token at a time: one 16-byte read of each CTA's sums
        const int quads = kFp4Rows / 4 / a.split, r0 = rank * (kFp4Rows / a.split);
        const uint32_t base = smem_u32(sm);
        for (int e = threadIdx.x; e < a.M * quads; e += kFp4Threads) {
            const int c = e / quads, row = r0 + 4 * (e % quads);
            const int64_t n = (int64_t)tile * kFp4Rows + row;
            if (n >= a.N) continue;  // (what is read is stored: no read is still under way at the barrier below)
            const uint32_t at = base + (uint32_t)(c * kFp4Rows + row) * 4;
            float4 v[kFp4MaxSplit];
#pragma unroll
            for (int r = 0; r < kFp4MaxSplit; ++r)
                v[r] = r < a.split ? ld_cluster_v4(map_rank(at, (uint32_t)r)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int r = 1; r < kFp4MaxSplit; ++r) v[0].x += v[r].x, v[0].y += v[r].y, v[0].z += v[r].z, v[0].w += v[r].w;
            const float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) fp4_store(a.y, c * a.ldy + n + i, fp4_scaled(o[i], g), a.ytype);
        }
        cluster_sync_relaxed();  // nobody reads this CTA's shared memory any more
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
}

}  // namespace bitnet

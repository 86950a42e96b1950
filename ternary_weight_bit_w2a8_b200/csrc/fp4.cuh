// fp4.cuh -- microscaled 4-bit floating point: quantisation, reading back and
// the tensor scale.
//
// Elements are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a
// byte with the even k in the low half.  MX: 32 elements along K share an e8m0
// scale (a power of two); NV: 16 share an e4m3 scale and the tensor an fp32
// scale g.  With z = fl32(x * fl32(1 / g)) and top = max |z| of a block:
//   MX: s = 2^(floor(log2 top) - 2), within 2^-127 .. 2^127 (2^-127 for top = 0)
//   NV: s = e4m3_rne_sat(fl32(top / 6))
//   element = e2m1_rne_sat(z / s)      (0 for s = 0)
// A block that holds a NaN or an infinity gets a NaN scale and elements 0, so
// whatever reads it gives NaN.  The definition rounds z once and the quotient
// once; the code below keeps that exact (see div_exact).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "fp4_plan.h"

namespace bitnet {

constexpr int kFp4TileBytes = 512;  // 128 rows x 4 blocks, one byte each

__host__ __device__ __forceinline__ int fp4_block(int format) { return format == BITNET_FP4_MX ? 32 : 16; }
__host__ __device__ __forceinline__ int64_t fp4_row_bytes(int64_t K) { return k_pad(K) / 2; }
// scale tiles of a 128-row band
__host__ __device__ __forceinline__ int64_t fp4_scale_tiles(int64_t K, int format) {
    return k_pad(K) / (4 * fp4_block(format));
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same where no memory is handed over: nobody leaves, or goes on, early.
__device__ __forceinline__ void cluster_sync_relaxed() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// ------------------------------------------------------------------ element types of x and y
template <int DT>
struct Fp4Type;
template <>
struct Fp4Type<BITNET_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float to_f(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T from_f(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Fp4Type<BITNET_FP16> {
    using T = __half;
    static __device__ __forceinline__ float to_f(T v) { return __half2float(v); }
    static __device__ __forceinline__ T from_f(float v) { return __float2half_rn(v); }
};
template <>
struct Fp4Type<BITNET_FP32> {
    using T = float;
    static __device__ __forceinline__ float to_f(T v) { return v; }
    static __device__ __forceinline__ T from_f(float v) { return v; }
};

// Pairs of fp32 numbers in one 64-bit register: an instruction works on both,
// rounding each as its single form does.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 32 bytes of a row as they are stored: 16 values, or 8 of fp32.
template <int DT>
struct Fp4Raw {
    static constexpr int kValues = 32 / (int)sizeof(typename Fp4Type<DT>::T);
    uint32_t w[8];
};
// From column k, zeros from column K on.  32 whole bytes in one load where
// `wide` (they start on a 32-byte boundary), else two of 16 bytes; in any case
// such a group starts on a 16-byte boundary.
template <int DT>
__device__ __forceinline__ Fp4Raw<DT> fp4_load32(const typename Fp4Type<DT>::T *__restrict__ row, int64_t k, int64_t K,
                                                 bool wide) {
    using T = typename Fp4Type<DT>::T;
    constexpr int kHalf = Fp4Raw<DT>::kValues / 2;
    Fp4Raw<DT> v;
    if (wide && k + 2 * kHalf <= K) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                       "=r"(v.w[7])
                     : "l"(row + k));
        return v;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t c = k + i * kHalf;
        if (c + kHalf <= K) {
            reinterpret_cast<uint4 *>(v.w)[i] = __ldg(reinterpret_cast<const uint4 *>(row + c));
        } else {
            alignas(16) T t[kHalf];
#pragma unroll
            for (int j = 0; j < kHalf; ++j) t[j] = c + j < K ? row[c + j] : T(0.0f);
            reinterpret_cast<uint4 *>(v.w)[i] = *reinterpret_cast<uint4 *>(t);
        }
    }
    return v;
}

__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<__nv_bfloat162 *>(&a)), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b, __half) {
    const __half2 m = __hmax2_nan(__habs2(*reinterpret_cast<__half2 *>(&a)), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}

// max |v| as fp32 bits: NaN, or infinity's bits, if one is among them.
template <int DT>
__device__ __forceinline__ uint32_t fp4_absmax(const Fp4Raw<DT> &v) {
    uint32_t top = 0;
    if constexpr (DT == BITNET_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = v.w[i] & 0x7fffffffu;
            top = b > top ? b : top;
        }
    } else {
        using T = typename Fp4Type<DT>::T;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = absmax2(v.w[i], top, T(0.0f));
        const uint16_t lo = (uint16_t)top, hi = (uint16_t)(top >> 16);  // magnitudes order as their bits do
        const uint16_t m = lo > hi ? lo : hi;
        top = __float_as_uint(Fp4Type<DT>::to_f(*reinterpret_cast<const T *>(&m))) & 0x7fffffffu;
    }
    return top;
}

template <int DT>
__device__ __forceinline__ float fp4_value(const Fp4Raw<DT> &v, int i) {
    return Fp4Type<DT>::to_f(reinterpret_cast<const typename Fp4Type<DT>::T *>(v.w)[i]);
}
// Values 2i and 2i + 1 as a pair of fp32.
template <int DT>
__device__ __forceinline__ uint64_t fp4_pair(const Fp4Raw<DT> &v, int i) {
    if constexpr (DT == BITNET_BF16)
        return (uint64_t)(v.w[i] & 0xffff0000u) << 32 | (v.w[i] << 16);
    else
        return f2_pack(fp4_value<DT>(v, 2 * i), fp4_value<DT>(v, 2 * i + 1));
}

// ------------------------------------------------------------------ rounding
// e4m3 of a >= 0 (finite), to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3_bits(float a) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(a));
    return r & 0xffu;
}

// The value of an e4m3 byte.
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __half2float(__ushort_as_half((uint16_t)(h & 0xffffu)));
}

// The value of an e8m0 byte: 2^(b - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : (b == 0u ? 0x00400000u : b << 23));
}

// Eight e2m1 codes (to nearest even, saturating at 6), the first in the low
// bits.
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&v)[4]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    return r;
}

// z / s rounded so that a comparison with any midpoint m of two e2m1 values
// comes out as it does for the exact quotient.  s has four significant bits
// and m three, so m s is an fp32 number: z is m s or at least one fp32 step
// from it, which moves the quotient by more than half a step of m (1.06 times
// that at least).  One residual correction of z * r (Markstein 1990), r within
// a step or two of 1 / s, reaches that: the residual z - q s is exact under
// fma, and what r is off enters only through its product with the residual.
// The same holds for top / 6 against the midpoints of e4m3 (five bits, 6 has
// two).
__device__ __forceinline__ float div_exact(float z, float s, float r) {
    const float q = __fmul_rn(z, r);
    return __fmaf_rn(__fmaf_rn(-q, s, z), r, q);
}

__device__ __forceinline__ float rcp_near(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

// Block scale from the bits of top = max |z| (an fp32 magnitude): its byte,
// and what quantising divides by.
struct Fp4Scale {
    uint32_t byte;
    float s, r;  // NV: the scale and about 1 / scale (0, 0 for a zero scale); MX: r = 1 / scale, exact
};

template <int FMT>
__device__ __forceinline__ Fp4Scale fp4_scale(uint32_t top) {
    Fp4Scale q;
    if (FMT == BITNET_FP4_MX) {
        // the exponent field holds floor(log2 top) + 127 (0 for subnormals,
        // which are below 2^-126: their scale is at the lower end as well)
        const int e = (int)(top >> 23) - 2;
        q.byte = top >= 0x7f800000u ? 255u : (uint32_t)(e < 0 ? 0 : e);
        q.s = 0.0f;
        // 2^(127 - byte): byte <= 252, so never subnormal
        q.r = top >= 0x7f800000u ? 0.0f : __uint_as_float((254u - q.byte) << 23);
    } else {
        q.byte = top >= 0x7f800000u ? 0x7fu : e4m3_bits(div_exact(__uint_as_float(top), 6.0f, 0.16666667f));
        const float s = e4m3_value(q.byte);
        const bool some = s > 0.0f;  // neither zero nor NaN
        q.s = some ? s : 0.0f;
        q.r = some ? rcp_near(s) : 0.0f;
    }
    return q;
}

// The codes of eight values x (in pairs) of a block: z = x * inv, then z / s.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_codes8(const uint64_t (&x)[4], float inv, const Fp4Scale &q, bool finite) {
    const uint64_t inv2 = f2_pack(inv, inv), r2 = f2_pack(q.r, q.r), ns2 = f2_pack(-q.s, -q.s);
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t z = f2_mul(x[i], inv2), t = f2_mul(z, r2);
        // MX: exact; NV: div_exact
        v[i] = f2_unpack(FMT == BITNET_FP4_MX ? t : f2_fma(f2_fma(t, ns2, z), r2, t));
    }
    const uint32_t c = e2m1x8(v);
    return finite ? c : 0u;
}

// ------------------------------------------------------------------ quantisation
// A CTA quantises a patch of ROWS rows x 256 k.  A lane takes 32 bytes of a row
// (16 values, 8 of fp32): one block of NV, half of one of MX, or half and a
// quarter; the lanes of a block share its maximum by shuffles.  A lane asks for
// up to four rows before it uses the first (13824 x 5120 bf16 into NV: 33 us,
// one row at a time 53; packed fp32 arithmetic is 3 of what is between).  Scale
// bytes are put together in shared memory, so that words of four go out; rows
// of the last band past the matrix get scale 0.  The CTAs start at the matrix's
// end: where the tensor scale has just read it, that is what L2 still holds
// (2 % for 13824 x 5120).  Patches of 32 rows where 64 would leave SMs idle:
// 997 x 6910 fp16 takes 6.6 us with 32, 7.5 with 64, 10.1 with 128, 13824 x
// 5120 bf16 36.3, 34.1 and 36.1.
//   ALIGNED: rows of x start on 16-byte boundaries.  Otherwise a warp reads a
// row's values in order, one to a lane, and shared memory turns them round.
template <int DT, int FMT, bool ALIGNED, int ROWS>
__global__ void __launch_bounds__(kThreads) fp4_quant_kernel(const typename Fp4Type<DT>::T *__restrict__ x,
                                                             int64_t rows, int64_t K, int64_t ldx,
                                                             const float *__restrict__ g, uint8_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales) {
    using T = typename Fp4Type<DT>::T;
    constexpr int B = FMT == BITNET_FP4_MX ? 32 : 16;
    constexpr int V = Fp4Raw<DT>::kValues;        // values of a lane
    constexpr int kLanes = kFp4PatchK / V;        // lanes of a row: 16 or 32
    constexpr int kTiles = kFp4PatchK / (4 * B);  // scale tiles of a patch: 2 or 4
    constexpr int kStep = kThreads / kLanes;      // rows that the CTA takes at once
    constexpr int kMost = ALIGNED ? 4 : 2, kAhead = ROWS / kStep < kMost ? ROWS / kStep : kMost;
    constexpr int kParts = kFp4TileRows / ROWS;   // patches of a 128-row band
    constexpr int kWords = ROWS / 32;             // 4-byte words of a tile's 16-byte row that a patch fills
    static_assert(ROWS == 32 || ROWS == 64, "rows of a patch");
    __shared__ uint32_t st[kTiles * 32 * kWords];
    __shared__ alignas(16) T turn[ALIGNED ? 1 : kStep * kFp4PatchK];
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int64_t patches_k = ceil_div(k_pad(K), kFp4PatchK);
    const int64_t block = gridDim.x - 1 - blockIdx.x, part = block / patches_k, pk = block % patches_k;
    const int64_t row_bytes = fp4_row_bytes(K), tiles = fp4_scale_tiles(K, FMT);
    const int64_t k = pk * kFp4PatchK + V * lane;
    const bool wide = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ldx * (int64_t)sizeof(T))) & 31) == 0;
    const int64_t left = rows - part * ROWS;
    const int nrows = (int)(left < 0 ? 0 : (left < ROWS ? left : ROWS));
    if (nrows < ROWS)
        for (int i = threadIdx.x; i < kTiles * 32 * kWords; i += kThreads) st[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const float inv = g != nullptr ? __frcp_rn(*g) : 1.0f;
    __syncthreads();
    x += part * ROWS * ldx;
    codes += part * ROWS * row_bytes + k / 2;
    const int at = (lane * V / (4 * B)) * 32 * kWords * 4 + (lane * V / B & 3);
    const bool stored = k / 2 < row_bytes;
    for (int r0 = group; r0 - group < nrows; r0 += kAhead * kStep) {  // (whole warps go on: they shuffle)
        Fp4Raw<DT> v[kAhead];
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (r0 + i * kStep < nrows) v[i] = fp4_load32<DT>(x + (r0 + i * kStep) * ldx, k, K, wide);
        } else {
            T t[kAhead][V];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int64_t c = pk * kFp4PatchK + j * kLanes + lane;
                    t[i][j] = r0 + i * kStep < nrows && c < K ? x[(r0 + i * kStep) * ldx + c] : T(0.0f);
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < V; ++j) turn[group * kFp4PatchK + j * kLanes + lane] = t[i][j];
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    reinterpret_cast<uint4 *>(v[i].w)[j] =
                        reinterpret_cast<const uint4 *>(turn + group * kFp4PatchK + V * lane)[j];
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kStep;
            // max |z| is fl32(max |x| * inv): rounding keeps order
            uint32_t top = r < nrows ? fp4_absmax<DT>(v[i]) : 0u;
            top = __float_as_uint(__fmul_rn(__uint_as_float(top), inv)) & 0x7fffffffu;
#pragma unroll
            for (int o = 1; o < B / V; o *= 2) {
                const uint32_t t = __shfl_xor_sync(0xffffffffu, top, o);
                top = t > top ? t : top;
            }
            if (r >= nrows) continue;
            const Fp4Scale q = fp4_scale<FMT>(top);
            uint32_t c[V / 8];
#pragma unroll
            for (int h = 0; h < V / 8; ++h) {
                uint64_t p[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = fp4_pair<DT>(v[i], 4 * h + j);
                c[h] = fp4_codes8<FMT>(p, inv, q, top < 0x7f800000u);
            }
            if (stored) {
                if constexpr (V == 16)
                    *reinterpret_cast<uint2 *>(codes + r * row_bytes) = make_uint2(c[0], c[1]);
                else
                    *reinterpret_cast<uint32_t *>(codes + r * row_bytes) = c[0];
            }
            if (lane % (B / V) == 0)
                reinterpret_cast<uint8_t *>(st)[at + ((r & 31) * kWords + (r >> 5)) * 4] = (uint8_t)q.byte;
        }
    }
    __syncthreads();
    // word w of tile row r of a tile: rows r + 32 w of the patch
    uint32_t *to = reinterpret_cast<uint32_t *>(scales + part / kParts * tiles * kFp4TileBytes) + part % kParts * kWords;
    for (int i = threadIdx.x; i < kTiles * 32; i += kThreads) {
        const int64_t t = pk * kTiles + i / 32;
        if (t >= tiles) continue;
        uint32_t *p = to + t * (kFp4TileBytes / 4) + (i & 31) * 4;
        if constexpr (kWords == 2)
            *reinterpret_cast<uint2 *>(p) = make_uint2(st[i * 2], st[i * 2 + 1]);
        else
            *p = st[i];
    }
}

// ------------------------------------------------------------------ reading back
// y[r, k] = round(fl32(element * scale) * g); element * scale is exact.

// The eight values of a word of codes as pairs of fp32.
__device__ __forceinline__ void e2m1_values8(uint32_t c, uint64_t (&v)[4]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[i] = f2_pack(f.x, f.y);
    }
}

// Two fp32 values as two of the type, packed (one of fp32 at a time).
template <int DT>
__device__ __forceinline__ uint32_t fp4_round2(float2 v) {
    uint32_t r;
    if (DT == BITNET_FP16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    return r;
}

// A CTA reads a patch of ROWS rows x 256 k; a lane takes 32 bytes of a row of y
// (16 values from 8 code bytes, 8 of fp32 from 4).  ALIGNED (rows of y start on
// 16-byte boundaries): stored as they are, at once where they start on a
// 32-byte boundary.  Otherwise the lanes of a row put them down in shared
// memory as 4-byte words that lie on 4-byte boundaries of y (shifted by one
// value where the row starts between two) and store those in order: 997 x 6910
// fp16 took 22 us with lanes that stored their own pairs.
template <int DT, int FMT, bool ALIGNED, int ROWS>
__global__ void __launch_bounds__(kThreads) fp4_dequant_kernel(const uint8_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales, int64_t rows,
                                                               int64_t K, const float *__restrict__ g,
                                                               typename Fp4Type<DT>::T *__restrict__ y, int64_t ldy) {
    using T = typename Fp4Type<DT>::T;
    constexpr int B = FMT == BITNET_FP4_MX ? 32 : 16;
    constexpr int V = Fp4Raw<DT>::kValues, kLanes = kFp4PatchK / V, kStep = kThreads / kLanes;
    constexpr int kAhead = ROWS / kStep < 4 ? ROWS / kStep : 4, kParts = kFp4TileRows / ROWS;
    constexpr int kRowWords = 8 * kLanes + kLanes;  // a word of padding after 8: lanes 8 words apart share no banks
    __shared__ uint32_t turn[ALIGNED ? 1 : kStep * kRowWords];
    const int64_t patches_k = ceil_div(k_pad(K), kFp4PatchK);
    const int64_t part = (int64_t)blockIdx.x / patches_k, pk = (int64_t)blockIdx.x % patches_k;
    const int64_t row_bytes = fp4_row_bytes(K), tiles = fp4_scale_tiles(K, FMT), k0 = pk * kFp4PatchK;
    const int64_t left = rows - part * ROWS;
    const int nrows = (int)(left < 0 ? 0 : (left < ROWS ? left : ROWS));
    const bool wide = ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(ldy * (int64_t)sizeof(T))) & 31) == 0;
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, k = V * lane;
    pdl_wait();
    pdl_launch_dependents();
    const float gs = g != nullptr ? *g : 1.0f;
    codes += part * ROWS * row_bytes + (k0 + k) / 2;
    scales += (part / kParts * tiles + (k0 + k) / (4 * B)) * kFp4TileBytes + part % kParts * (ROWS / 32 * 4) + (k / B & 3);
    y += part * ROWS * ldy + k0;
    const int cols = (int)(K - k0 < kFp4PatchK ? K - k0 : kFp4PatchK);
    uint32_t *words = turn + group * kRowWords;
    for (int r0 = group; r0 - group < nrows; r0 += kAhead * kStep) {  // (whole warps go on: they shuffle)
        uint32_t c[kAhead][V / 8], sb[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kStep;
            if (r < nrows && k < cols) {
#pragma unroll
                for (int h = 0; h < V / 8; ++h)
                    c[i][h] = *reinterpret_cast<const uint32_t *>(codes + r * row_bytes + 4 * h);
                sb[i] = scales[16 * (r & 31) + 4 * (r >> 5)];
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kStep;
            if (ALIGNED && (r >= nrows || k >= cols)) continue;
            const float s = FMT == BITNET_FP4_MX ? e8m0_value(sb[i]) : e4m3_value(sb[i]);
            uint32_t w[8];
#pragma unroll
            for (int h = 0; h < V / 8; ++h) {
                uint64_t e[4];
                e2m1_values8(c[i][h], e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = f2_unpack(f2_mul(f2_mul(e[j], f2_pack(s, s)), f2_pack(gs, gs)));
                    if constexpr (sizeof(T) == 4)
                        w[2 * j] = __float_as_uint(f.x), w[2 * j + 1] = __float_as_uint(f.y);
                    else
                        w[4 * h + j] = fp4_round2<DT>(f);
                }
            }
            const T *t = reinterpret_cast<const T *>(w);
            T *yr = y + r * ldy;
            if constexpr (ALIGNED) {
                if (wide && k + V <= cols) {
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(yr + k), "r"(w[0]),
                                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                 : "memory");
                    continue;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (k + (h + 1) * (V / 2) <= cols) {
                        reinterpret_cast<uint4 *>(yr + k)[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
                    } else {
#pragma unroll
                        for (int j = h * (V / 2); j < (h + 1) * (V / 2); ++j)
                            if (k + j < cols) yr[k + j] = t[j];
                    }
                }
            } else {
                constexpr int kPer = 4 / (int)sizeof(T);  // values of a word
                // word q holds values kPer q - odd and the next
                const int odd = kPer == 2 ? (int)(reinterpret_cast<uintptr_t>(yr) >> 1 & 1) : 0;
                const uint32_t before = __shfl_up_sync(0xffffffffu, w[7], 1);
                __syncwarp();  // the words of the row before have been read
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    words[9 * lane + j] = odd ? __funnelshift_l(j > 0 ? w[j > 0 ? j - 1 : 0] : before, w[j], 16) : w[j];
                __syncwarp();
                if (r < nrows) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int q = lane + j * kLanes, e = kPer * q - odd;
                        const uint32_t v = words[q + (q >> 3)];
                        if (e >= 0 && e + kPer <= cols) {
                            *reinterpret_cast<uint32_t *>(yr + e) = v;
                        } else if (kPer == 2) {  // the row's first or last value alone
                            const uint16_t half = (uint16_t)(e < 0 ? v >> 16 : v);
                            const int at = e < 0 ? 0 : e;
                            if (at < cols) yr[at] = *reinterpret_cast<const T *>(&half);
                        }
                    }
                    // the patch's last value, where the words end one before it
                    if (odd && lane == kLanes - 1 && cols == kFp4PatchK) yr[kFp4PatchK - 1] = t[V - 1];
                }
            }
        }
    }
}

// ------------------------------------------------------------------ tensor scale
// g = max(fl32(max |x| / 2688), 2^-126) over the finite values of x (2688 =
// 6 * 448: the largest value the NV format holds at g = 1; the lower end keeps
// 1 / g finite).  Rounding keeps order, so g is also the largest of the CTAs'
// own values: they meet in an atomic maximum of the bits (positive floats order
// as their bits do; a maximum does not depend on the order), g having been set
// to 0 by a launch before.  What kFp4ScaleCluster CTAs take in one round of
// loads (256 KB) is one cluster instead: the first CTA reads the others' values
// and stores g, and there is no launch before (16 x 2560 bf16: 3.6 us of host
// time and 2.5 of the GPU's, not 5.9 and 2.4).  A warp takes a piece of a
// row at a time, four 32-byte loads to a lane; the values before the row's
// first 32-byte boundary and behind its last are taken one by one.
__global__ void fp4_clear_kernel(float *g) {
    pdl_wait();
    pdl_launch_dependents();
    *g = 0.0f;
}

constexpr int kFp4ScaleLoads = 4;
constexpr int kFp4ScaleCluster = 8;
template <int DT>
constexpr int kFp4ScalePiece = Fp4Raw<DT>::kValues * 32 * kFp4ScaleLoads;

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) fp4_tensor_scale_kernel(const typename Fp4Type<DT>::T *__restrict__ x,
                                                                    int64_t rows, int64_t K, int64_t ldx, float *g) {
    using T = typename Fp4Type<DT>::T;
    constexpr int V = Fp4Raw<DT>::kValues;
    __shared__ uint32_t red[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t per_row = ceil_div(K, kFp4ScalePiece<DT>), total = rows * per_row;
    pdl_wait();
    pdl_launch_dependents();
    uint32_t top = 0;
    auto one = [&](T v) {
        const uint32_t b = __float_as_uint(Fp4Type<DT>::to_f(v)) & 0x7fffffffu;
        top = b < 0x7f800000u && b > top ? b : top;
    };
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < total; i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t row = i / per_row, piece = i - row * per_row;
        const T *xr = x + row * ldx;
        int64_t head = (int64_t)((0 - reinterpret_cast<uintptr_t>(xr)) & 31) / (int64_t)sizeof(T);
        if (head > K) head = K;
        const int64_t end = head + (K - head) / V * V;  // of the whole 32-byte groups
        const int64_t k0 = head + piece * kFp4ScalePiece<DT> + V * lane;
        Fp4Raw<DT> v[kFp4ScaleLoads];
#pragma unroll
        for (int j = 0; j < kFp4ScaleLoads; ++j) {
            const int64_t k = k0 + j * 32 * V;
            if (k < end) {
                v[j] = fp4_load32<DT>(xr, k, K, true);
            } else {
#pragma unroll
                for (int w = 0; w < 8; ++w) v[j].w[w] = 0;
            }
        }
        if (piece == 0) {
            if (lane < head) one(xr[lane]);
            if (end + lane < K) one(xr[end + lane]);
        }
#pragma unroll
        for (int j = 0; j < kFp4ScaleLoads; ++j) {
            const uint32_t t = fp4_absmax<DT>(v[j]);
            if (t < 0x7f800000u) {
                top = t > top ? t : top;
            } else {  // the finite ones among them
#pragma unroll
                for (int e = 0; e < V; ++e) one(reinterpret_cast<const T *>(v[j].w)[e]);
            }
        }
    }
    top = block_reduce(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; }, red);
    const bool cluster = gridDim.x <= kFp4ScaleCluster;  // launched as one
    __shared__ uint32_t mine;
    if (cluster && gridDim.x > 1) {
        if (threadIdx.x == 0) mine = top;
        cluster_sync();
    }
    if (threadIdx.x == 0 && !(cluster && blockIdx.x > 0)) {
        if (cluster)
            for (uint32_t r = 1; r < gridDim.x; ++r) {
                const uint32_t t = ld_cluster_u32(map_rank((uint32_t)__cvta_generic_to_shared(&mine), r));
                top = t > top ? t : top;
            }
        const float v = __fdiv_rn(__uint_as_float(top), 2688.0f);
        const float s = v > 1.17549435e-38f ? v : 1.17549435e-38f;
        if (cluster)
            *g = s;
        else
            atomicMax(reinterpret_cast<uint32_t *>(g), __float_as_uint(s));
    }
    // nobody leaves while its value may be read (g has been stored from them before the reader arrives)
    if (cluster && gridDim.x > 1) cluster_sync_relaxed();
}

}  // namespace bitnet

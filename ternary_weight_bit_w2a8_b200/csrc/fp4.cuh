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

namespace bitnet {

constexpr int kFp4TileRows = 128;   // rows of a scale tile
constexpr int kFp4TileBytes = 512;  // 128 rows x 4 blocks, one byte each

__host__ __device__ __forceinline__ int fp4_block(int format) { return format == BITNET_FP4_MX ? 32 : 16; }
__host__ __device__ __forceinline__ int64_t fp4_row_bytes(int64_t K) { return k_pad(K) / 2; }
// scale tiles of a 128-row band
__host__ __device__ __forceinline__ int64_t fp4_scale_tiles(int64_t K, int format) {
    return k_pad(K) / (4 * fp4_block(format));
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

// 8 consecutive values of a row from column k, zeros from column K on.  `vec`:
// every such group of the row starts on a 16-byte boundary.
template <int DT>
__device__ __forceinline__ void fp4_load8(const typename Fp4Type<DT>::T *__restrict__ row, int64_t k, int64_t K,
                                          bool vec, float (&v)[8]) {
    using T = typename Fp4Type<DT>::T;
    if (vec && k + 8 <= K) {
        alignas(16) T t[8];
#pragma unroll
        for (int i = 0; i < (int)sizeof(t) / 16; ++i)
            reinterpret_cast<uint4 *>(t)[i] = __ldg(reinterpret_cast<const uint4 *>(row + k) + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Fp4Type<DT>::to_f(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < K ? Fp4Type<DT>::to_f(row[k + i]) : 0.0f;
    }
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

// Eight e2m1 codes (to nearest even, saturating at 6), v[0] in the low bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// z / s rounded so that a comparison with any midpoint m of two e2m1 values
// comes out as it does for the exact quotient.  s has four significant bits
// and m three, so m s is an fp32 number: z is m s or at least one fp32 step
// from it, which moves the quotient by more than half a step of m.  One
// residual correction of z * r, r = fl32(1 / s), reaches that: the residual
// z - q s is exact under fma, and q + residual * r is off by a step only
// where the quotient is no midpoint.
__device__ __forceinline__ float div_exact(float z, float s, float r) {
    const float q = __fmul_rn(z, r);
    return __fmaf_rn(__fmaf_rn(-q, s, z), r, q);
}

// Block scale from the bits of top = max |z| (an fp32 magnitude): its byte,
// and what quantising divides by.
struct Fp4Scale {
    uint32_t byte;
    float s, r;  // NV: the scale and fl32(1 / scale) (0, 0 for a zero scale); MX: r = 1 / scale, exact
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
        q.byte = top >= 0x7f800000u ? 0x7fu : e4m3_bits(__fdiv_rn(__uint_as_float(top), 6.0f));
        q.s = e4m3_value(q.byte);
        q.r = q.s > 0.0f ? __frcp_rn(q.s) : 0.0f;
        if (!(q.s > 0.0f)) q.s = 0.0f;
    }
    return q;
}

template <int FMT>
__device__ __forceinline__ uint32_t fp4_codes8(const float (&z)[8], const Fp4Scale &q, bool finite) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = FMT == BITNET_FP4_MX ? __fmul_rn(z[i], q.r) : div_exact(z[i], q.s, q.r);
    const uint32_t c = e2m1x8(v);
    return finite ? c : 0u;
}

// ------------------------------------------------------------------ quantisation
// A CTA quantises a patch of 128 rows x 256 k, so that it writes whole scale
// tiles: a warp takes rows w, w + 8, ..., a lane 8 consecutive k of a row (one
// 16-byte load of 16-bit values); the lanes of a block share its maximum by
// shuffles; scale bytes are put together in shared memory.  The rows of the
// last band past the matrix get scale 0.
constexpr int kFp4PatchK = 256;

template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) fp4_quant_kernel(const typename Fp4Type<DT>::T *__restrict__ x,
                                                             int64_t rows, int64_t K, int64_t ldx,
                                                             const float *__restrict__ g, uint8_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales) {
    constexpr int B = FMT == BITNET_FP4_MX ? 32 : 16;
    constexpr int kTiles = kFp4PatchK / (4 * B);  // scale tiles of a patch: 2 or 4
    __shared__ alignas(16) uint8_t st[kTiles * kFp4TileBytes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t patches_k = ceil_div(k_pad(K), kFp4PatchK);
    const int64_t band = (int64_t)blockIdx.x / patches_k, pk = (int64_t)blockIdx.x % patches_k;
    const int64_t row_bytes = fp4_row_bytes(K), tiles = fp4_scale_tiles(K, FMT);
    const int64_t k = pk * kFp4PatchK + 8 * lane;
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ldx * (int64_t)sizeof(*x))) & 15) == 0;
    for (int i = threadIdx.x; i < kTiles * kFp4TileBytes / 4; i += kThreads) reinterpret_cast<uint32_t *>(st)[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const float inv = g != nullptr ? __frcp_rn(*g) : 1.0f;
    __syncthreads();
    const int64_t left = rows - band * kFp4TileRows;
    const int nrows = (int)(left < kFp4TileRows ? left : kFp4TileRows);
    const int tile = lane * 8 / (4 * B), col = (lane * 8 / B) & 3;
    for (int r = warp; r < nrows; r += kThreads / 32) {
        const int64_t row = band * kFp4TileRows + r;
        float z[8];
        fp4_load8<DT>(x + row * ldx, k, K, vec, z);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] = __fmul_rn(z[i], inv);
            const uint32_t b = __float_as_uint(z[i]) & 0x7fffffffu;
            top = b > top ? b : top;
        }
#pragma unroll
        for (int o = 1; o < B / 8; o *= 2) {
            const uint32_t t = __shfl_xor_sync(0xffffffffu, top, o);
            top = t > top ? t : top;
        }
        const Fp4Scale q = fp4_scale<FMT>(top);
        const uint32_t c = fp4_codes8<FMT>(z, q, top < 0x7f800000u);
        if (k / 2 < row_bytes) *reinterpret_cast<uint32_t *>(codes + row * row_bytes + k / 2) = c;
        if (lane % (B / 8) == 0) st[tile * kFp4TileBytes + 16 * (r & 31) + 4 * (r >> 5) + col] = (uint8_t)q.byte;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTiles * kFp4TileBytes / 16; i += kThreads) {
        const int64_t t = pk * kTiles + i / (kFp4TileBytes / 16);
        if (t < tiles)
            reinterpret_cast<uint4 *>(scales + (band * tiles + t) * kFp4TileBytes)[i % (kFp4TileBytes / 16)] =
                reinterpret_cast<const uint4 *>(st)[i];
    }
}

// ------------------------------------------------------------------ reading back
// y[r, k] = round(fl32(element * scale) * g); element * scale is exact.  A lane
// takes 8 consecutive k of a row: 4 code bytes, one scale byte.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) fp4_dequant_kernel(const uint8_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales, int64_t rows,
                                                               int64_t K, const float *__restrict__ g,
                                                               typename Fp4Type<DT>::T *__restrict__ y, int64_t ldy) {
    using T = typename Fp4Type<DT>::T;
    constexpr int B = FMT == BITNET_FP4_MX ? 32 : 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t patches_k = ceil_div(k_pad(K), kFp4PatchK);
    const int64_t band = (int64_t)blockIdx.x / patches_k, pk = (int64_t)blockIdx.x % patches_k;
    const int64_t row_bytes = fp4_row_bytes(K), tiles = fp4_scale_tiles(K, FMT);
    const int64_t k = pk * kFp4PatchK + 8 * lane;
    const bool vec = ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(ldy * (int64_t)sizeof(T))) & 15) == 0;
    pdl_wait();
    pdl_launch_dependents();
    if (k >= K) return;
    const float gs = g != nullptr ? *g : 1.0f;
    const int64_t left = rows - band * kFp4TileRows;
    const int nrows = (int)(left < kFp4TileRows ? left : kFp4TileRows);
    const uint8_t *sp = scales + (band * tiles + k / (4 * B)) * kFp4TileBytes + (k / B & 3);
    for (int r = warp; r < nrows; r += kThreads / 32) {
        const int64_t row = band * kFp4TileRows + r;
        const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + row * row_bytes + k / 2);
        const uint32_t sb = sp[16 * (r & 31) + 4 * (r >> 5)];
        const float s = FMT == BITNET_FP4_MX ? e8m0_value(sb) : e4m3_value(sb);
        alignas(16) T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the three magnitude bits as exponent and mantissa of an fp32
            // number stand for the e2m1 value times 2^-126 (subnormals included)
            const uint32_t n = c >> (4 * i);
            const float e = __uint_as_float((n & 7u) << 22) * 8.507059173023462e37f;  // 2^126
            const float v = __uint_as_float(__float_as_uint(e) | ((n & 8u) << 28));
            t[i] = Fp4Type<DT>::from_f(__fmul_rn(__fmul_rn(v, s), gs));
        }
        T *yp = y + row * ldy + k;
        if (vec && k + 8 <= K) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(t) / 16; ++i) reinterpret_cast<uint4 *>(yp)[i] = reinterpret_cast<uint4 *>(t)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < K) yp[i] = t[i];
        }
    }
}

// ------------------------------------------------------------------ tensor scale
// g = max(fl32(max |x| / 2688), 2^-126) over the finite values of x (2688 =
// 6 * 448: the largest value the NV format holds at g = 1; the lower end keeps
// 1 / g finite).  Two launches: a maximum per CTA, then one CTA over those;
// maxima do not depend on any order.
constexpr int kFp4ScaleMaxBlocks = 1184;

template <int DT>
__global__ void __launch_bounds__(kThreads) fp4_absmax_kernel(const typename Fp4Type<DT>::T *__restrict__ x,
                                                              int64_t rows, int64_t K, int64_t ldx,
                                                              uint32_t *__restrict__ partial) {
    __shared__ uint32_t red[32];
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ldx * (int64_t)sizeof(*x))) & 15) == 0;
    const int64_t per_row = ceil_div(K, 8), total = rows * per_row;
    pdl_wait();
    pdl_launch_dependents();
    uint32_t top = 0;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / per_row;
        float v[8];
        fp4_load8<DT>(x + row * ldx, 8 * (i - row * per_row), K, vec, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
            top = b < 0x7f800000u && b > top ? b : top;
        }
    }
    top = block_reduce(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; }, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = top;
}

__global__ void __launch_bounds__(kThreads) fp4_tensor_scale_kernel(const uint32_t *__restrict__ partial, int n,
                                                                    float *__restrict__ g) {
    __shared__ uint32_t red[32];
    pdl_wait();
    pdl_launch_dependents();
    uint32_t top = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) top = partial[i] > top ? partial[i] : top;
    top = block_reduce(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; }, red);
    if (threadIdx.x == 0) {
        const float v = __fdiv_rn(__uint_as_float(top), 2688.0f);
        *g = v > 1.17549435e-38f ? v : 1.17549435e-38f;
    }
}

}  // namespace bitnet

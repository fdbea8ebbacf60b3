// Microscaled (MX) blocks on the device: 32 values along K share one
// power-of-two scale (an E8M0 byte b, 2^(b - 127), 255 for NaN) and are kept
// as E2M1 codes (4 bits, two per byte, the even value in the low nibble) or
// E4M3 codes (8 bits).  Scales lie in tiles of 128 rows x 4 blocks, 512
// bytes: the byte of (row r, block b) is 16·(r % 32) + 4·(r % 128 / 32) +
// b % 4 of tile (r / 128, b / 4), tiles of one row block in K order.  That is
// the order in which the tensor cores take block scales, so a product copies
// tiles straight to tensor memory.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace q4mm {

constexpr int kMxBlock = 32;        // values per scale
constexpr int kMxPadK = 128;        // K is padded to a multiple of this
constexpr int kMxTileRows = 128;    // rows of a scale tile
constexpr int kMxTileBytes = 512;   // bytes of a scale tile (128 rows x 4 blocks)

__host__ __device__ constexpr int mx_padded(int K) { return (K + kMxPadK - 1) / kMxPadK * kMxPadK; }

// The largest of three magnitudes; a NaN stays one.
__device__ __forceinline__ float mx_max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Scale byte of a block whose largest magnitude has the float bits
// `amax_bits`: biased exponent of 2^(floor(log2 amax) - emax).  The float's
// own exponent field is floor(log2 amax) + 127 for a normal amax and 0 below,
// where the result is 0 either way.  255 (NaN) where the block holds an
// infinity or a NaN, whose bits compare above every finite magnitude.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, int emax) {
    const int e = (int)(amax_bits >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - emax, 0);
}

// 1 / scale as a float, exact: 2^(127 - b) for b <= 252.
__device__ __forceinline__ float mx_inverse(uint32_t b) { return __uint_as_float((254u - min(b, 253u)) << 23); }

// The scale itself: b = 0 is the subnormal 2^-127, b = 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

// Eight scaled values to codes, round to nearest even, cut at the largest
// code: one word of E2M1 (value i in nibble i) ...
__device__ __forceinline__ uint32_t mx_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// ... or two words of E4M3 (value i in byte i).
__device__ __forceinline__ uint32_t mx_e4m3x4(float v0, float v1, float v2, float v3) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    return r;
}

// Two codes back to values (exact in fp16, hence in fp32): byte k of four
// E2M1 pairs, or half k of two E4M3 pairs.
template <int k>
__device__ __forceinline__ float2 mx_from_e2m1x2(uint32_t bytes) {
    uint32_t h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
        : "=r"(h)
        : "r"(bytes), "n"(k));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
template <int k>
__device__ __forceinline__ float2 mx_from_e4m3x2(uint32_t bytes) {
    uint32_t h;
    asm("{\n\t.reg .b16 b0, b1;\n\tmov.b32 {b0, b1}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b%2;\n\t}"
        : "=r"(h)
        : "r"(bytes), "n"(k));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Element types of the unquantised side.
__device__ __forceinline__ float mx_float(float v) { return v; }
__device__ __forceinline__ float mx_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float mx_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T mx_from_float(float v);
template <>
__device__ __forceinline__ float mx_from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half mx_from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 mx_from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two values rounded to a 16-bit type, the lower in the low half.
template <class T>
__device__ __forceinline__ uint32_t mx_pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t mx_pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t mx_pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace q4mm

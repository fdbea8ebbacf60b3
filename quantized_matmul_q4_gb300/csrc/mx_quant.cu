// MX quantisation and what feeds it (sm_103a): plain quantisation, SwiGLU,
// residual addition with RMS norm, and the way back to values.
//
//   mx_quantize   v = x
//   mx_swiglu     v = gate / (1 + e^-gate) · up
//   mx_rmsnorm    h = x + residual, v = h · (mean_k h² + eps)^-1/2 · g, h written back
//
// each followed by q[k] = round(v[k] / s) in blocks of 32 with
// s = 2^(floor(log2 max |v|) - emax).  Everything between the loads and the
// one rounding to codes is fp32 (the sum of squares and the norm too); v / s
// is exact, a multiplication by a power of two, so a code has the single
// rounding of its conversion.  h is rounded once to its type; the norm takes
// the unrounded sum.
//
// All move 2 to 12 bytes per value and are meant to be bound by HBM.  A lane
// takes 8 consecutive values (16 bytes of a 16-bit type, 32 of fp32), a block
// is 4 lanes, so the block's maximum is two shuffles and the codes of a warp's
// 256 values are one contiguous store.  What else runs per value decides
// whether 16-bit inputs keep up with HBM (152 SMs issue some 75 lane
// instructions per value at 2 bytes per value), hence the packed arithmetic:
// magnitudes of 16-bit inputs are compared two at a time, products and
// conversions run on pairs, no index is divided, and the scale bytes of four
// rows change places by three shuffles instead of eight.
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace q4mm {

namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// Eight consecutive values of a row as they lie in memory, zeros past K.
template <class T>
struct Raw8 {
    uint32_t w[4];  // pairs, the lower value in the low half
};
template <>
struct Raw8<float> {
    uint32_t w[8];
};

// Words m / 32 onwards of c, shifted right by m % 32 bits: kOut words from bit
// m of the kIn given, m a multiple of 16 below 128, alike in the whole warp.
template <int kOut, int kIn>
__device__ __forceinline__ void words_from_bit(const uint32_t (&c)[kIn], int m, uint32_t (&out)[kOut]) {
    uint32_t u[kIn - 1], t[kIn - 3];
#pragma unroll
    for (int i = 0; i < kIn - 1; ++i) u[i] = m & 32 ? c[i + 1] : c[i];
#pragma unroll
    for (int i = 0; i < kIn - 3; ++i) t[i] = m & 64 ? u[i + 2] : u[i];
#pragma unroll
    for (int i = 0; i < kOut; ++i) out[i] = i + 1 < kIn - 3 ? __funnelshift_r(t[i], t[i + 1], m & 16) : t[i];
}

// Eight values on their way; several can be before the first is used.
// kVec: rows aligned to eight values and K a multiple of 8, so the eight are
// all inside or all outside.  Otherwise load<true> loads the 16-byte granules
// that hold them, which take() shifts: at the row's ends they reach up to 15
// bytes over it, so only where another row lies on that side (wide).
// load<false> loads the values one by one (8192 x 4095 bf16 to 8-bit codes:
// 26.4 us with that alone, 22.9 so).
template <bool kVec, class T>
struct Fetch8 {
    static constexpr int kWords = sizeof(T) * 2;
    uint32_t c[kVec ? kWords : kWords + 4];

    template <bool kWide>
    __device__ __forceinline__ void load(const T *row, int col, int K) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + col);
        if constexpr (kVec || kWide) {
            const int skip = kVec ? 0 : (int)(at & 15), have = min(8, K - col) * (int)sizeof(T);  // bytes
            const uint4 *from = reinterpret_cast<const uint4 *>(at - skip);
#pragma unroll
            for (int i = 0; i < (kVec ? kWords : kWords + 4); i += 4) {
                uint4 a = make_uint4(0u, 0u, 0u, 0u);
                if (have > 0 && (kVec || 4 * i < skip + have)) a = from[i / 4];
                c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (sizeof(T) == 4) {
                    c[i] = col + i < K ? reinterpret_cast<const uint32_t *>(row)[col + i] : 0u;
                } else {
                    const uint32_t b = col + i < K ? reinterpret_cast<const uint16_t *>(row)[col + i] : 0u;
                    c[i / 2] = i & 1 ? c[i / 2] | b << 16 : b;
                }
            }
#pragma unroll
            for (int i = kWords; i < kWords + 4; ++i) c[i] = 0u;
        }
    }
    __device__ __forceinline__ void take(const T *row, int col, int K, bool wide, Raw8<T> &r) const {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) r.w[i] = c[i];
        } else {
            const int skip = wide ? (int)(reinterpret_cast<uintptr_t>(row + col) & 15) : 0;
            const int have = min(8, K - col) * (int)sizeof(T);
            words_from_bit(c, 8 * skip, r.w);
            if (have < 8 * (int)sizeof(T)) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    if (4 * i >= have) r.w[i] = 0u;
                    if (sizeof(T) == 2 && 4 * i + 2 == have) r.w[i] &= 0xFFFFu;
                }
            }
        }
    }
};

__device__ __forceinline__ void to_float(const Raw8<float> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void to_float(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void to_float(const Raw8<__half> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

// Eight values of one row alone, of which nothing outside may be read.
template <bool kVec, class T>
__device__ __forceinline__ void load8(const T *row, int col, int K, float (&v)[8]) {
    if constexpr (!kVec) {
        if (reinterpret_cast<uintptr_t>(row) % 16 == 0 && col + 8 <= K) return load8<true>(row, col, K, v);
    }
    Fetch8<kVec, T> f;
    Raw8<T> r;
    f.template load<false>(row, col, K);
    f.take(row, col, K, false, r);
    to_float(r, v);
}

// Stores eight values per lane, nothing past K.  Every lane of the warp takes
// part, with columns eight apart.  Without kVec the row starts anywhere: a
// lane writes the 16-byte granules that begin among its own values, the last
// of them with the next lane's first values, and single values only at the
// warp's and the row's ends.
template <bool kVec, class T>
__device__ __forceinline__ void store8(T *row, int col, int K, const float (&v)[8]) {
    constexpr int kWords = sizeof(T) * 2, kEach = 16 / sizeof(T);  // values of a granule
    uint32_t d[kWords];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = mx_pack2<T>(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (kVec) {
        if (col >= K) return;
        if constexpr (sizeof(T) == 4) {
            // One 32-byte store: a sector is written at once, not in halves.
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + col), "r"(d[0]),
                         "r"(d[1]), "r"(d[2]), "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7])
                         : "memory");
        } else {
            *reinterpret_cast<uint4 *>(row + col) = make_uint4(d[0], d[1], d[2], d[3]);
        }
    } else {
        const int lane = threadIdx.x & 31;
        const int skip = (int)(reinterpret_cast<uintptr_t>(row + col) & 15) / (int)sizeof(T);
        const int head = skip ? kEach - skip : 0;  // values before the first granule that begins here
        uint32_t e[kWords + 4], g[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) e[i] = d[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[kWords + i] = __shfl_down_sync(kFull, d[i], 1);
        words_from_bit(e, 8 * (int)sizeof(T) * head, g);
        auto one = [&](int j) {
            if (col + j < K) row[col + j] = mx_from_float<T>(v[j]);
        };
        // The values before the first granule are the previous lane's to
        // write where it writes that granule whole.
        const bool mine = lane == 0 || col + head > K;
#pragma unroll
        for (int j = 0; j < kEach - 1; ++j)
            if (j < head && mine) one(j);
#pragma unroll
        for (int i = 0; i < 8 / kEach; ++i) {
            const int first = head + i * kEach;
            const bool whole = first + kEach <= 8 || lane != 31;
            if (whole && col + first + kEach <= K) {
                *reinterpret_cast<uint4 *>(row + col + first) =
                    make_uint4(g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j >= first && j < first + kEach) one(j);
            }
        }
    }
}

// The same from the values as they lie in memory.
template <class T>
__device__ __forceinline__ uint32_t block_amax(const Raw8<T> &r, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        return mx_block_amax(v);
    } else {
        // Two at a time: 16-bit magnitudes as packed numbers of their type.
        using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
        auto mag = [&](int i) {
            const uint32_t w = r.w[i] & 0x7FFF7FFFu;
            return *reinterpret_cast<const T2 *>(&w);
        };
        T2 m = __hmax2_nan(__hmax2_nan(mag(0), mag(1)), __hmax2_nan(mag(2), mag(3)));
        m = __hmax2_nan(m, __shfl_xor_sync(kFull, m, 1));
        m = __hmax2_nan(m, __shfl_xor_sync(kFull, m, 2));
        return __float_as_uint(mx_float(__hmax_nan(m.x, m.y)));
    }
}
__device__ __forceinline__ uint32_t block_amax(const Raw8<float> &, const float (&v)[8]) { return mx_block_amax(v); }

// The exchange of scale bytes.  Four lanes hold a block; the four such groups
// g = lane / 4 % 4 of a half warp hold, in byte i of `p`, the scale of their
// block of row (or column chunk) i.  Afterwards group g holds row g's word:
// the bytes of its four blocks in order.  p of group g ^ k comes by shuffle k;
// byte g of it goes to byte g ^ k of the word.
struct ByteExchange {
    uint32_t s01, s23, s;
    __device__ __forceinline__ explicit ByteExchange(int lane) {
        const uint32_t g = (lane >> 2) & 3;
        s01 = g << (4 * g) | (4 + g) << (4 * (g ^ 1));
        s23 = g << (4 * (g ^ 2)) | (4 + g) << (4 * (g ^ 3));
        s = g & 2 ? 0x3254u : 0x7610u;  // bytes g and g ^ 1 from the first pair
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t p) const {
        const uint32_t a = __byte_perm(p, __shfl_xor_sync(kFull, p, 4), s01);
        const uint32_t b = __byte_perm(__shfl_xor_sync(kFull, p, 8), __shfl_xor_sync(kFull, p, 12), s23);
        return __byte_perm(a, b, s);
    }
};

// x / (1 + e^-x) of two values, to 9·2^-24, for x >= kSiluFar.  e^-x is 2^t,
// t = -x·log2 e; the product's rounding, and log2 e's own, would cost |t|
// units in the last place, so t = hi + lo and 2^t = 2^hi + 2^hi·lo·ln 2 (with
// expf and an exact quotient 4099 x 11008 bf16 takes 53.6 us instead of 35.7,
// where the bytes alone take 33).  Infinities above and NaN pass through the
// quotient; below kSiluFar its reciprocal would be subnormal, which is flushed.
constexpr float kSiluFar = -87.f;  // 1 + e^87 < 2^126
__device__ __forceinline__ float2 silu2(float2 x) {
    const float2 c = make_float2(fminf(x.x, 100.f), fminf(x.y, 100.f));
    const float2 l2e = make_float2(-1.44269504f, -1.44269504f);    // -log2 e, and what it lacks
    const float2 rest = make_float2(-1.92596303e-8f, -1.92596303e-8f);
    const float2 ln2 = make_float2(0.693147181f, 0.693147181f);
    const float2 hi = __fmul2_rn(c, l2e);
    const float2 lo = __fmul2_rn(ffma2(c, rest, ffma2(c, l2e, make_float2(-hi.x, -hi.y))), ln2);
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(hi.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(hi.y));
    e = __fadd2_rn(ffma2(e, lo, e), make_float2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
    return __fmul2_rn(x, e);
}

// x / (1 + e^-x) · up for x < kSiluFar, where 1 + e^-x is e^-x to 2^-125: so
// x·e^x·up.  e^x falls out of fp32's normal range there, while the product
// with a large up need not: e^x is taken as e^(x + 100)·c·c, c = e^-50, and no
// product on the way overflows or loses bits that the last one keeps (x + 100
// is exact).  -inf gives NaN, as the quotient does.
__device__ __forceinline__ float silu_far(float x, float up) {
    constexpr float c = 1.92874985e-22f;
    return (x * expf(x + 100.f)) * (up * c) * c;
}

__device__ __forceinline__ float min3(float a, float b, float c) {  // of NaN and a number the number
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// silu(v)·u of eight values into v.  Products of gates below kSiluFar are not
// to be used without kFar, which puts them right.
template <bool kFar>
__device__ __forceinline__ void swiglu8(float (&v)[8], const float (&u)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float2 f = __fmul2_rn(silu2(make_float2(v[j], v[j + 1])), make_float2(u[j], u[j + 1]));
        if constexpr (kFar) {
            if (v[j] < kSiluFar) f.x = silu_far(v[j], u[j]);
            if (v[j + 1] < kSiluFar) f.y = silu_far(v[j + 1], u[j + 1]);
        }
        v[j] = f.x, v[j + 1] = f.y;
    }
}

// Whether any of the gates seen lies below kSiluFar.  In bfloat16 the words
// are compared as they lie, four values at a time: as unsigned numbers those
// below it are the largest (and NaN with a sign, which may pass for one).
// 4099 x 11008 to 8 bits: 36.0 -> 35.7 us; float16 is slower so (35.7 -> 38.4).
template <class T>
struct FarGates {
    float least = 0.f;
    uint32_t most = 0u;
    __device__ __forceinline__ void see(const Raw8<T> &r, const float (&v)[8]) {
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            most = __vimax3_u16x2(__vimax3_u16x2(most, r.w[0], r.w[1]), r.w[2], r.w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j += 2) least = min3(least, v[j], v[j + 1]);
        }
    }
    __device__ __forceinline__ bool any() const {
        return least < kSiluFar || max(most >> 16, most & 0xFFFFu) > 0xC2AEu;  // -87
    }
};

// One warp per 256 columns of the four rows r, r + 32, r + 64, r + 96 of a
// 128-row block, whose scale words are 16 contiguous bytes of a tile (four
// rows also keep four independent loads in flight per lane).  Rows past the
// last one get zero scale bytes and no codes.  blockIdx.x: 32 row groups per
// 128-row block; blockIdx.y and the warp: the column chunk.
// CTAs per SM that the registers have to allow: SwiGLU 4, and 3 unaligned
// (4099 x 11008 bf16: 46.7 -> 35.7 us; 8192 x 4095: 50.9 -> 43.3);
// else 4 unaligned (8192 x 4095 bf16 to 8-bit codes: 26.7 -> 22.5).
template <class T, bool kVec, bool kSwiGLU>
__global__ void __launch_bounds__(256, kSwiGLU ? (kVec ? 4 : 3) : (kVec ? 1 : 4))
    mx_quantize_kernel(const T *__restrict__ x, long long x_stride, const T *__restrict__ up, long long up_stride,
                       uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int K, int rows, int bits) {
    const int Kp = mx_padded(K), nkt = Kp / kMxPadK;
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int r = blockIdx.x & 31;
    const unsigned block = blockIdx.x >> 5;
    const int col = 256 * c + 8 * lane;
    const size_t code_row = (size_t)Kp * bits / 8;
    const long long row0 = (long long)block * kMxTileRows + r;
    pdl_wait();
    if (2 * c >= nkt) return;
    // Neither the first row nor the last one is among the four; K >= 8: a
    // neighbour is 16 bytes at least.
    const bool wide = row0 > 0 && K >= 8 && ((rows - 1 - row0) % 32 != 0 || rows - row0 > kMxTileRows);
    Fetch8<kVec, T> fx[4];
    const T *px = x + row0 * x_stride;
    auto width = [&](int i) { return row0 + 32 * i < rows ? K : 0; };
    auto load4 = [&](const T *from, long long stride, Fetch8<kVec, T>(&f)[4]) {
        if (kVec || wide) {  // (one branch around all of them keeps them side by side)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i].template load<true>(from + 32 * i * stride, col, width(i));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i].template load<false>(from + 32 * i * stride, col, width(i));
        }
    };
    load4(px, x_stride, fx);
    uint32_t p = 0;
    uint8_t *pc = codes + row0 * code_row;
    if constexpr (kSwiGLU) {
        Fetch8<kVec, T> fu[4];
        const T *pu = up + row0 * up_stride;
        load4(pu, up_stride, fu);
        FarGates<T> gates;
        auto row = [&](auto far, int i, const Fetch8<kVec, T> &gx, const Fetch8<kVec, T> &gu) {
            Raw8<T> rx, ru;
            float v[8], u[8];
            gx.take(px + 32 * i * x_stride, col, width(i), wide, rx);
            gu.take(pu + 32 * i * up_stride, col, width(i), wide, ru);
            to_float(rx, v);
            to_float(ru, u);
            if constexpr (!decltype(far)::value) gates.see(rx, v);
            swiglu8<decltype(far)::value>(v, u);
            return mx_quantize8(v, mx_block_amax(v), bits, pc + 32 * i * code_row, col, row0 + 32 * i < rows ? Kp : 0)
                   << (8 * i);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) p |= row(std::false_type{}, i, fx[i], fu[i]);
        // Gates below kSiluFar are rare: a warp that has met one reads its
        // four rows again.  (A branch for each row instead: 38 us on 4099 x
        // 11008 bf16, against 35.7.)
        if (__any_sync(kFull, gates.any())) {
            p = 0;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                Fetch8<kVec, T> gx, gu;
                if (kVec || wide) {
                    gx.template load<true>(px + 32 * i * x_stride, col, width(i));
                    gu.template load<true>(pu + 32 * i * up_stride, col, width(i));
                } else {
                    gx.template load<false>(px + 32 * i * x_stride, col, width(i));
                    gu.template load<false>(pu + 32 * i * up_stride, col, width(i));
                }
                p |= row(std::true_type{}, i, gx, gu);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Raw8<T> rx;
            float v[8];
            fx[i].take(px + 32 * i * x_stride, col, width(i), wide, rx);
            to_float(rx, v);
            p |= mx_quantize8(v, block_amax(rx, v), bits, pc + 32 * i * code_row, col, row0 + 32 * i < rows ? Kp : 0)
                 << (8 * i);
        }
    }
    const uint32_t w = ByteExchange(lane)(p);
    const int kt = 2 * c + (lane >> 4);
    if ((lane & 3) == 0 && kt < nkt)
        *reinterpret_cast<uint32_t *>(scales + ((size_t)block * nkt + kt) * kMxTileBytes + 16 * r + (lane & 12)) = w;
}

struct RmsArgs {
    const void *x, *residual, *weight;
    void *h;
    long long x_stride, residual_stride, h_stride;
    uint8_t *codes, *scales;
    float eps;
    int K, rows, bits;
    bool weight_f32;
};

// One CTA per row.  A thread keeps its kVals groups of 8 values of h in
// registers between the sum of squares and the quantisation, so x and the
// residual are read once; kVals = 0 (rows too long for that) reads and adds
// them again, from L2.  More values per thread cost a single row some latency
// and spread the fixed work (the reduction, indexes, scale words) of many
// rows over more values.
template <class T, bool kVec, int kVals>
__global__ void __launch_bounds__(1024) mx_rmsnorm_kernel(const RmsArgs a) {
    __shared__ float partial[32];
    const int K = a.K, Kp = mx_padded(K), nkt = Kp / kMxPadK;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const long long row = blockIdx.x;
    const int step = 8 * blockDim.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
    T *h = a.h ? static_cast<T *>(a.h) + row * a.h_stride : nullptr;
    pdl_wait();
    if (row >= a.rows) {
        // The CTAs past the last row write zero scale bytes for the rest of
        // its 128-row block, a thread per word (one row of 4096: 4.4 -> 2.2
        // us against leaving it to the row's own CTA).
        const int first = (a.rows - 1) / kMxTileRows * kMxTileRows, here = a.rows - first;
        uint8_t *tiles = a.scales + (size_t)(first / kMxTileRows) * nkt * kMxTileBytes;
        const int words = (kMxTileRows - here) * nkt, all = (int)(gridDim.x - a.rows) * blockDim.x;
        for (int i = (int)(row - a.rows) * blockDim.x + threadIdx.x; i < words; i += all) {
            const int p = here + i / nkt, kt = i % nkt;
            *reinterpret_cast<uint32_t *>(tiles + (size_t)kt * kMxTileBytes + 16 * (p & 31) + 4 * (p >> 5)) = 0u;
        }
        return;
    }
    constexpr int kKept = kVals > 0 ? kVals : 1;
    const bool wide = row > 0 && row < a.rows - 1 && K >= 8;
    // Groups are loaded four at a time at most, x and residual together; two
    // unaligned, whose granules would not fit the registers (8192 x 4095 bf16:
    // 62.1 -> 61.0 us).
    auto load_h = [&](int c0, float (&v)[kKept][8]) {
        constexpr int kAhead = kVec || kKept < 2 ? kKept : 2;
#pragma unroll
        for (int i0 = 0; i0 < kKept; i0 += kAhead) {
            auto col = [&](int i) { return c0 + (i0 + i) * step + 8 * (int)threadIdx.x; };
            Fetch8<kVec, T> fx[kAhead], fr[kAhead];
            auto load_all = [&](const T *from, Fetch8<kVec, T>(&f)[kAhead]) {
                if (kVec || wide) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) f[i].template load<true>(from, col(i), K);
                } else {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) f[i].template load<false>(from, col(i), K);
                }
            };
            load_all(x, fx);
            if (res) load_all(res, fr);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                Raw8<T> r;
                fx[i].take(x, col(i), K, wide, r);
                to_float(r, v[i0 + i]);
                if (res) {
                    float u[8];
                    fr[i].take(res, col(i), K, wide, r);
                    to_float(r, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i0 + i][j] += u[j];
                }
            }
        }
    };
    float v[kKept][8];
    float2 sums = make_float2(0.f, 0.f);
    auto add_squares = [&]() {
#pragma unroll
        for (int i = 0; i < kKept; ++i)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 f = make_float2(v[i][j], v[i][j + 1]);
                sums = ffma2(f, f, sums);
            }
    };
    auto load_g = [&](int c0, float (&g)[8]) {
        if (a.weight_f32) {
            load8<kVec>(static_cast<const float *>(a.weight), c0 + 8 * threadIdx.x, K, g);
        } else {
            load8<kVec>(static_cast<const T *>(a.weight), c0 + 8 * threadIdx.x, K, g);
        }
    };
    float g0[8];
    if constexpr (kVals > 0) {
        load_h(0, v);
        // With one group a thread, the form for few rows, the chain of
        // latencies is what counts: the weight is loaded beside x.
        if constexpr (kVals == 1) load_g(0, g0);
        add_squares();
    } else {
        for (int c0 = 0; c0 < K; c0 += step) {
            load_h(c0, v);
            add_squares();
        }
    }
    float sum = warp_sum(sums.x + sums.y);
    if (lane == 0) partial[warp] = sum;
    __syncthreads();
    // Every warp adds the partial sums in the same order: one barrier, and
    // the same bits everywhere.
    sum = warp_sum(lane < nwarps ? partial[lane] : 0.f);
    const float norm = rsqrtf(sum / (float)K + a.eps);
    uint8_t *codes_row = a.codes + (size_t)row * Kp * a.bits / 8;
    // Byte 16·(r % 32) + 4·(r % 128 / 32) of the row's tiles.
    uint8_t *scale_row = a.scales + (size_t)(row / kMxTileRows) * nkt * kMxTileBytes + 16 * (row & 31) +
                         4 * ((row & 127) >> 5);
    // Writes h, quantises a group of 8 values per thread, returns its scale byte.
    auto finish = [&](int c0, float (&u)[8]) {
        const int col = c0 + 8 * threadIdx.x;
        if (h) store8<kVec>(h, col, K, u);
        float g[8];
        if constexpr (kVals == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = g0[j];
        } else {
            load_g(c0, g);
        }
        // Past K the values are zeros and so is the weight; an infinite norm
        // or a NaN must not reach the padding.
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = u[j] * norm * g[j];
        if (kVec ? col >= K : col + 8 > K) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j >= K) u[j] = 0.f;
        }
        return mx_quantize8(u, mx_block_amax(u), a.bits, codes_row, col, Kp);
    };
    const ByteExchange exchange(lane);
    const int g4 = (lane >> 2) & 3;  // which group's word this lane writes
    if constexpr (kVals > 0) {
        uint32_t p = 0;
#pragma unroll
        for (int i = 0; i < kVals; ++i) p |= finish(i * step, v[i]) << (8 * i);
        const uint32_t w = exchange(p);
        const int kt = (g4 * step + 256 * warp) / kMxPadK + (lane >> 4);
        if ((lane & 3) == 0 && g4 < kVals && kt < nkt)
            *reinterpret_cast<uint32_t *>(scale_row + (size_t)kt * kMxTileBytes) = w;
    } else {
        for (int c0 = 0; c0 < Kp; c0 += step) {
            load_h(c0, v);
            const uint32_t w = exchange(finish(c0, v[0]));
            const int kt = (c0 + 256 * warp) / kMxPadK + (lane >> 4);
            if ((lane & 15) == 0 && kt < nkt) *reinterpret_cast<uint32_t *>(scale_row + (size_t)kt * kMxTileBytes) = w;
        }
    }
}

// Codes and scales back to values, with the quantising kernel's division of
// the work: the scale words of a warp's four rows are one 16-byte load.
template <class T, bool kVec, int kBits>
__global__ void __launch_bounds__(256)
    mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, T *__restrict__ y,
                         long long y_stride, int K, int rows) {
    const int Kp = mx_padded(K), nkt = Kp / kMxPadK;
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int r = blockIdx.x & 31;
    const unsigned block = blockIdx.x >> 5;
    const int col = 256 * c + 8 * lane, kt = 2 * c + (lane >> 4);
    const long long row0 = (long long)block * kMxTileRows + r;
    pdl_wait();
    if (2 * c >= nkt || row0 >= rows) return;
    const bool inside = kt < nkt;  // (the warp's second half may lie past the last tile)
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (inside)
        w = *reinterpret_cast<const uint4 *>(scales + ((size_t)block * nkt + kt) * kMxTileBytes + 16 * r);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
    const size_t code_row = (size_t)Kp * kBits / 8;
    const uint8_t *p = codes + row0 * code_row + (size_t)col * kBits / 8;
    uint2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = make_uint2(0u, 0u);
        if (inside && row0 + 32 * i < rows) {
            if (kBits == 4)
                q[i].x = *reinterpret_cast<const uint32_t *>(p + 32 * i * code_row);
            else
                q[i] = *reinterpret_cast<const uint2 *>(p + 32 * i * code_row);
        }
    }
    T *py = y + row0 * y_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (row0 + 32 * i >= rows) break;
        const float s = mx_scale((word[i] >> (8 * ((lane >> 2) & 3))) & 0xFFu);
        float2 f[4];
        if constexpr (kBits == 4) {
            f[0] = mx_from_e2m1x2<0>(q[i].x), f[1] = mx_from_e2m1x2<1>(q[i].x);
            f[2] = mx_from_e2m1x2<2>(q[i].x), f[3] = mx_from_e2m1x2<3>(q[i].x);
        } else {
            f[0] = mx_from_e4m3x2<0>(q[i].x), f[1] = mx_from_e4m3x2<1>(q[i].x);
            f[2] = mx_from_e4m3x2<0>(q[i].y), f[3] = mx_from_e4m3x2<1>(q[i].y);
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = __fmul2_rn(f[j], make_float2(s, s));
            v[2 * j] = t.x, v[2 * j + 1] = t.y;
        }
        store8<kVec>(py + 32 * i * y_stride, col, K, v);
    }
}

// Every row starts on a multiple of eight values (of 16 or 32 bytes).
template <class T>
bool rows_aligned(const void *p, long long stride) {
    return reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0 && stride % 8 == 0;
}

// Warps of 256 columns by groups of four rows: up to 8 column chunks per CTA.
struct RowGrid {
    dim3 grid, block;
};
RowGrid row_grid(int K, int rows) {
    const unsigned chunks = (unsigned)(mx_padded(K) + 255) / 256;
    const unsigned warps = chunks < 8 ? chunks : 8;
    const unsigned groups = (unsigned)(((long long)rows + kMxTileRows - 1) / kMxTileRows * 32);
    return RowGrid{dim3(groups, (chunks + warps - 1) / warps), dim3(32 * warps)};
}

template <class T>
cudaError_t quantize_t(const LaunchCtx &c, const MxQuantizeArgs &a) {
    const RowGrid g = row_grid(a.K, a.rows);
    const bool vec = a.K % 8 == 0 && rows_aligned<T>(a.x, a.x_stride) && (!a.up || rows_aligned<T>(a.up, a.up_stride));
    auto kernel = a.up ? (vec ? mx_quantize_kernel<T, true, true> : mx_quantize_kernel<T, false, true>)
                       : (vec ? mx_quantize_kernel<T, true, false> : mx_quantize_kernel<T, false, false>);
    return launch_kernel(c, kernel, g.grid, g.block, 0, static_cast<const T *>(a.x), a.x_stride,
                         static_cast<const T *>(a.up), a.up_stride, a.codes, a.scales, a.K, a.rows, a.bits);
}

template <class T>
cudaError_t rmsnorm_t(const LaunchCtx &c, const MxRmsnormArgs &a) {
    const bool vec = a.K % 8 == 0 && rows_aligned<T>(a.x, a.x_stride) &&
                     (!a.residual || (rows_aligned<T>(a.residual, a.residual_stride))) &&
                     (!a.h || rows_aligned<T>(a.h, a.h_stride)) && reinterpret_cast<uintptr_t>(a.weight) % 32 == 0;
    const RmsArgs k{a.x, a.residual, a.weight, a.h, a.x_stride, a.residual_stride, a.h_stride, a.codes, a.scales,
                    a.eps, a.K, a.rows, a.bits, a.weight_f32};
    const int Kp = mx_padded(a.K);
    // Values per thread: the fewest that 1024 threads allow, a group of 8, for
    // fp32 and while there are no more rows than SMs (one row of 4096: 2.1
    // us); for many rows of a 16-bit type four groups, where they leave four
    // warps.  8192 x 4096 bf16 with a residual: 52.0, 38.1, 37.6 us with one,
    // two, four groups; 4096 x 4096 fp32: 34.9 with one, 35.9 with two, 37.8
    // with four.  Unaligned rows have more fixed work: from 1024 on two groups
    // where the aligned ones have one (4096 x 4095 fp32: 52.3, 38.7, 42.7 with
    // one, two, four; 30000 x 1117 fp16: 84.8, 81.3, 110; 20000 x 513 fp32:
    // 33.9, 38.4, 41.9; 8192 x 4095 bf16: 81.3, 61.3, 58.7).
    int vals = 1;
    if (a.rows > c.num_sms && sizeof(T) == 2) vals = Kp >= 4096 ? 4 : Kp >= 2048 ? 2 : 1;
    if (a.rows > c.num_sms && !vec && vals == 1 && Kp >= 1024) vals = 2;
    while (vals < 4 && Kp > 8 * 1024 * vals) vals *= 2;
    const bool kept = Kp <= 8 * 1024 * vals;
    int threads = kept ? (Kp / 8 + vals - 1) / vals : 1024;
    threads = (threads + 31) / 32 * 32;
    auto pick = [&](auto v1, auto v2, auto v4, auto v0) { return !kept ? v0 : vals == 1 ? v1 : vals == 2 ? v2 : v4; };
    auto kernel = vec ? pick(mx_rmsnorm_kernel<T, true, 1>, mx_rmsnorm_kernel<T, true, 2>,
                             mx_rmsnorm_kernel<T, true, 4>, mx_rmsnorm_kernel<T, true, 0>)
                      : pick(mx_rmsnorm_kernel<T, false, 1>, mx_rmsnorm_kernel<T, false, 2>,
                             mx_rmsnorm_kernel<T, false, 4>, mx_rmsnorm_kernel<T, false, 0>);
    // CTAs for the padding's scale bytes, two words a thread.
    const int words = (kMxTileRows - 1 - (a.rows - 1) % kMxTileRows) * (Kp / kMxPadK);
    const int padding = (words + 2 * threads - 1) / (2 * threads);
    return launch_kernel(c, kernel, dim3((unsigned)a.rows + padding), dim3(threads), 0, k);
}

template <class T>
cudaError_t dequantize_t(const LaunchCtx &c, const MxDequantizeArgs &a) {
    const RowGrid g = row_grid(a.K, a.rows);
    const bool vec = a.K % 8 == 0 && rows_aligned<T>(a.y, a.y_stride);
    auto kernel = a.bits == 4 ? (vec ? mx_dequantize_kernel<T, true, 4> : mx_dequantize_kernel<T, false, 4>)
                              : (vec ? mx_dequantize_kernel<T, true, 8> : mx_dequantize_kernel<T, false, 8>);
    return launch_kernel(c, kernel, g.grid, g.block, 0, a.codes, a.scales, static_cast<T *>(a.y), a.y_stride, a.K,
                         a.rows);
}

}  // namespace

cudaError_t launch_mx_quantize(const LaunchCtx &c, MxType type, const MxQuantizeArgs &a) {
    return type == MxType::kF32   ? quantize_t<float>(c, a)
           : type == MxType::kF16 ? quantize_t<__half>(c, a)
                                  : quantize_t<__nv_bfloat16>(c, a);
}

cudaError_t launch_mx_rmsnorm(const LaunchCtx &c, MxType type, const MxRmsnormArgs &a) {
    return type == MxType::kF32   ? rmsnorm_t<float>(c, a)
           : type == MxType::kF16 ? rmsnorm_t<__half>(c, a)
                                  : rmsnorm_t<__nv_bfloat16>(c, a);
}

cudaError_t launch_mx_dequantize(const LaunchCtx &c, MxType type, const MxDequantizeArgs &a) {
    return type == MxType::kF32   ? dequantize_t<float>(c, a)
           : type == MxType::kF16 ? dequantize_t<__half>(c, a)
                                  : dequantize_t<__nv_bfloat16>(c, a);
}

}  // namespace q4mm

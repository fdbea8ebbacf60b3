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
// kVec: rows aligned to eight values and K a multiple of 8, so the eight are
// all inside or all outside.
template <class T>
struct Raw8 {
    uint32_t w[4];  // pairs, the lower value in the low half
};
template <>
struct Raw8<float> {
    float v[8];
};

template <bool kVec, class T>
__device__ __forceinline__ void load8(const T *row, int col, int K, Raw8<T> &r) {
    if constexpr (sizeof(T) == 4) {
        if (kVec) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (col < K) {
                a = *reinterpret_cast<const float4 *>(row + col);
                b = *reinterpret_cast<const float4 *>(row + col + 4);
            }
            r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
            r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = col + i < K ? row[col + i] : 0.f;
        }
    } else {
        if (kVec) {
            uint4 a = make_uint4(0u, 0u, 0u, 0u);
            if (col < K) a = *reinterpret_cast<const uint4 *>(row + col);
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        } else {
            const unsigned short *p = reinterpret_cast<const unsigned short *>(row);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = col + 2 * i < K ? p[col + 2 * i] : 0u;
                const uint32_t hi = col + 2 * i + 1 < K ? p[col + 2 * i + 1] : 0u;
                r.w[i] = lo | hi << 16;
            }
        }
    }
}

__device__ __forceinline__ void to_float(const Raw8<float> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.v[i];
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

template <bool kVec, class T>
__device__ __forceinline__ void load8(const T *row, int col, int K, float (&v)[8]) {
    Raw8<T> r;
    load8<kVec>(row, col, K, r);
    to_float(r, v);
}

template <bool kVec, class T>
__device__ __forceinline__ void store8(T *row, int col, int K, const float (&v)[8]) {
    if constexpr (kVec) {
        if (col < K) {
            if constexpr (sizeof(T) == 4) {
                // One 32-byte store: a sector is written at once, not in halves.
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + col), "f"(v[0]),
                             "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                             : "memory");
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = mx_pack2<T>(v[2 * i], v[2 * i + 1]);
                *reinterpret_cast<uint4 *>(row + col) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < K) row[col + i] = mx_from_float<T>(v[i]);
    }
}

// Float bits of the largest magnitude of eight values, and of the 32 of a
// block over its four lanes; NaN where one of them is.
__device__ __forceinline__ uint32_t block_amax(const float (&v)[8]) {
    const float a = mx_max3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2]));
    const float b = mx_max3(fabsf(v[3]), fabsf(v[4]), fabsf(v[5]));
    float m = mx_max3(a, b, fabsf(v[6]));
    m = mx_max3(m, fabsf(v[7]), __shfl_xor_sync(kFull, mx_max3(m, fabsf(v[7]), m), 1));
    return __float_as_uint(mx_max3(m, __shfl_xor_sync(kFull, m, 2), m));
}

template <class T>
__device__ __forceinline__ uint32_t block_amax(const Raw8<T> &r, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        return block_amax(v);
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
__device__ __forceinline__ uint32_t block_amax(const Raw8<float> &, const float (&v)[8]) { return block_amax(v); }

// Quantises the block of `amax` (float bits) that this lane's eight values
// belong to, stores their codes (nothing where col >= Kp) and returns the
// block's scale byte.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t amax, int bits, uint8_t *codes_row, int col,
                                              int Kp) {
    const uint32_t b = mx_scale_byte(amax, bits == 4 ? 2 : 8);
    const float2 inv = make_float2(mx_inverse(b), mx_inverse(b));
    float s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), inv);
        s[2 * i] = f.x, s[2 * i + 1] = f.y;
    }
    if (col < Kp) {
        // The codes under a NaN scale are zeros.
        if (bits == 4) {
            *reinterpret_cast<uint32_t *>(codes_row + (col >> 1)) = b == 255 ? 0u : mx_e2m1x8(s);
        } else {
            const uint32_t lo = mx_e4m3x4(s[0], s[1], s[2], s[3]), hi = mx_e4m3x4(s[4], s[5], s[6], s[7]);
            *reinterpret_cast<uint2 *>(codes_row + col) = make_uint2(b == 255 ? 0u : lo, b == 255 ? 0u : hi);
        }
    }
    return b;
}

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

// x / (1 + e^-x) of two values, to about 6 units in the last place.  e^-x is
// 2^t, t = -x·log2 e; the product's rounding, and log2 e's own, would cost
// |t| units in the last place, so t = hi + lo and 2^t = 2^hi + 2^hi·lo·ln 2
// (with expf and an exact quotient 4099 x 11008 bf16 takes 42.6 us instead of
// 36.3, where the bytes alone take 33).
// Past |x| = 88.7 e^-x is 0 or beyond the range of the approximate quotient,
// which is then a zero; infinities and NaN pass through the quotient.
__device__ __forceinline__ float2 silu2(float2 x) {
    const float2 c = make_float2(fminf(fmaxf(x.x, -88.7f), 100.f), fminf(fmaxf(x.y, -88.7f), 100.f));
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

// One warp per 256 columns of the four rows r, r + 32, r + 64, r + 96 of a
// 128-row block, whose scale words are 16 contiguous bytes of a tile (four
// rows also keep four independent loads in flight per lane).  Rows past the
// last one get zero scale bytes and no codes.  blockIdx.x: 32 row groups per
// 128-row block; blockIdx.y and the warp: the column chunk.
template <class T, bool kVec, bool kSwiGLU>
__global__ void __launch_bounds__(256, kSwiGLU ? 4 : 1)  // (four CTAs: 37.5 -> 36.3 us on 4099 x 11008 bf16)
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
    Raw8<T> raw[4];
    const T *px = x + row0 * x_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) load8<kVec>(px + 32 * i * x_stride, col, row0 + 32 * i < rows ? K : 0, raw[i]);
    uint32_t p = 0;
    uint8_t *pc = codes + row0 * code_row;
    if constexpr (kSwiGLU) {
        Raw8<T> rup[4];
        const T *pu = up + row0 * up_stride;
#pragma unroll
        for (int i = 0; i < 4; ++i) load8<kVec>(pu + 32 * i * up_stride, col, row0 + 32 * i < rows ? K : 0, rup[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8], u[8];
            to_float(raw[i], v);
            to_float(rup[i], u);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 f =
                    __fmul2_rn(silu2(make_float2(v[j], v[j + 1])), make_float2(u[j], u[j + 1]));
                v[j] = f.x, v[j + 1] = f.y;
            }
            p |= quantize8(v, block_amax(v), bits, pc + 32 * i * code_row, col, row0 + 32 * i < rows ? Kp : 0)
                 << (8 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
            to_float(raw[i], v);
            p |= quantize8(v, block_amax(raw[i], v), bits, pc + 32 * i * code_row, col, row0 + 32 * i < rows ? Kp : 0)
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
    // Groups are loaded four at a time at most, x and residual together.
    auto load_h = [&](int c0, float (&v)[kKept][8]) {
        Raw8<T> rx[kKept], rr[kKept];
#pragma unroll
        for (int i = 0; i < kKept; ++i) load8<kVec>(x, c0 + i * step + 8 * threadIdx.x, K, rx[i]);
        if (res) {
#pragma unroll
            for (int i = 0; i < kKept; ++i) load8<kVec>(res, c0 + i * step + 8 * threadIdx.x, K, rr[i]);
        }
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            to_float(rx[i], v[i]);
            if (res) {
                float u[8];
                to_float(rr[i], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += u[j];
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
        return quantize8(u, block_amax(u), a.bits, codes_row, col, Kp);
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
    if (kt >= nkt || row0 >= rows) return;
    const uint4 w = *reinterpret_cast<const uint4 *>(scales + ((size_t)block * nkt + kt) * kMxTileBytes + 16 * r);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
    const size_t code_row = (size_t)Kp * kBits / 8;
    const uint8_t *p = codes + row0 * code_row + (size_t)col * kBits / 8;
    uint2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = make_uint2(0u, 0u);
        if (row0 + 32 * i < rows) {
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
    // with four.
    int vals = 1;
    if (a.rows > c.num_sms && sizeof(T) == 2) vals = Kp >= 4096 ? 4 : Kp >= 2048 ? 2 : 1;
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

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
// All are bound by HBM: 2 to 8 bytes read and 0.5 to 1 written per value
// against some 20 instructions.  A lane takes 8 consecutive values (one
// 16-byte load of 16-bit values, one 32-byte load of fp32), a block is 4
// lanes, so the block's maximum is two shuffles and the codes of a warp's 256
// values are one contiguous store.
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace q4mm {

namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// Eight consecutive values of a row, zeros past K.  kVec: 16-byte aligned
// rows and K a multiple of 8, so the eight are all inside or all outside.
template <bool kVec, class T>
__device__ __forceinline__ void load8(const T *row, int col, int K, float (&v)[8]) {
    if constexpr (kVec) {
        if (col < K) {
            if constexpr (sizeof(T) == 4) {
                const float4 a = *reinterpret_cast<const float4 *>(row + col);
                const float4 b = *reinterpret_cast<const float4 *>(row + col + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
                const uint4 a = *reinterpret_cast<const uint4 *>(row + col);
                const T *e = reinterpret_cast<const T *>(&a);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = mx_float(e[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < K ? mx_float(row[col + i]) : 0.f;
    }
}

template <bool kVec, class T>
__device__ __forceinline__ void store8(T *row, int col, int K, const float (&v)[8]) {
    if constexpr (kVec) {
        if (col < K) {
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4 *>(row + col) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(row + col + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                uint4 a;
                T *e = reinterpret_cast<T *>(&a);
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = mx_from_float<T>(v[i]);
                *reinterpret_cast<uint4 *>(row + col) = a;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < K) row[col + i] = mx_from_float<T>(v[i]);
    }
}

// Quantises a warp's 256 values (8 per lane from column col = c0 + 8·lane on;
// col may lie past Kp, where nothing is stored), stores the codes of the row
// and returns, in every lane, the scale word of its half: the four scale
// bytes of columns c0 + 128·(lane / 16) onwards.
__device__ __forceinline__ uint32_t quantize_warp(const float (&v)[8], int bits, uint8_t *codes_row, int col, int Kp) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    m = max(m, __shfl_xor_sync(kFull, m, 2));
    const uint32_t b = mx_scale_byte(m, bits == 4 ? 2 : 8);
    const float inv = mx_inverse(b);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = b == 255 ? 0.f : v[i] * inv;  // the codes under a NaN scale are zeros
    if (col < Kp) {
        if (bits == 4) {
            *reinterpret_cast<uint32_t *>(codes_row + (col >> 1)) = mx_e2m1x8(s);
        } else {
            *reinterpret_cast<uint2 *>(codes_row + col) =
                make_uint2(mx_e4m3x4(s[0], s[1], s[2], s[3]), mx_e4m3x4(s[4], s[5], s[6], s[7]));
        }
    }
    const int lane = threadIdx.x & 31;
    uint32_t w = b << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(kFull, w, 4);
    w |= __shfl_xor_sync(kFull, w, 8);
    return w;
}

// x / (1 + e^-x), by the quotient's definition; e^-x overflows to infinity
// for x below about -88, where the quotient is -0.
__device__ __forceinline__ float silu(float x) { return x / (1.f + expf(-x)); }

// One warp per item: 256 columns of the four rows r, r + 32, r + 64, r + 96
// of a 128-row block, whose scale words are 16 contiguous bytes of a tile
// (four rows also keep four independent loads in flight per lane).  Rows past
// the last one get zero scale bytes and no codes.
template <class T, bool kVec, bool kSwiGLU>
__global__ void __launch_bounds__(256)
    mx_quantize_kernel(const T *__restrict__ x, long long x_stride, const T *__restrict__ up, long long up_stride,
                       uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int K, int rows, int bits,
                       long long items) {
    const int Kp = mx_padded(K), nkt = Kp / kMxPadK, chunks = (Kp + 255) / 256;
    const long long item = blockIdx.x * 8LL + (threadIdx.x >> 5);
    pdl_wait();
    if (item >= items) return;
    const int lane = threadIdx.x & 31;
    const int c = (int)(item % chunks);
    const long long rr = item / chunks;  // 32 row groups per 128-row block
    const int r = (int)(rr & 31);
    const long long block = rr >> 5;
    const int col = 256 * c + 8 * lane;
    const size_t code_row = (size_t)Kp * bits / 8;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long row = block * kMxTileRows + r + 32 * i;
        if (row < rows) {
            load8<kVec>(x + row * x_stride, col, K, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
    }
    if constexpr (kSwiGLU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long row = block * kMxTileRows + r + 32 * i;
            if (row < rows) {
                float u[8];
                load8<kVec>(up + row * up_stride, col, K, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = silu(v[i][j]) * u[j];
            }
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long row = block * kMxTileRows + r + 32 * i;
        // (A row past the end passes Kp = 0: its zero block stores nothing.)
        w[i] = quantize_warp(v[i], bits, codes + (row < rows ? row : 0) * code_row, col, row < rows ? Kp : 0);
    }
    const int kt = 2 * c + (lane >> 4);
    if ((lane & 15) == 0 && kt < nkt)
        *reinterpret_cast<uint4 *>(scales + ((size_t)block * nkt + kt) * kMxTileBytes + 16 * r) =
            make_uint4(w[0], w[1], w[2], w[3]);
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
// them again, from L2.
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
    auto load_h = [&](int col, float (&v)[8]) {
        load8<kVec>(x, col, K, v);
        if (res) {
            float r[8];
            load8<kVec>(res, col, K, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += r[j];
        }
    };
    constexpr int kKept = kVals > 0 ? kVals : 1;
    float v[kKept][8];
    float sum = 0.f;
    if constexpr (kVals > 0) {
#pragma unroll
        for (int i = 0; i < kVals; ++i) load_h(i * step + 8 * threadIdx.x, v[i]);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    } else {
        for (int c0 = 0; c0 < K; c0 += step) {
            load_h(c0 + 8 * threadIdx.x, v[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(v[0][j], v[0][j], sum);
        }
    }
    sum = warp_sum(sum);
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
    auto finish = [&](int c0, float (&u)[8]) {
        const int col = c0 + 8 * threadIdx.x;
        if (h) store8<kVec>(h, col, K, u);
        float g[8];
        if (a.weight_f32) {
            load8<kVec>(static_cast<const float *>(a.weight), col, K, g);
        } else {
            load8<kVec>(static_cast<const T *>(a.weight), col, K, g);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = col + j < K ? u[j] * norm * g[j] : 0.f;
        const uint32_t w = quantize_warp(u, a.bits, codes_row, col, Kp);
        const int kt = (c0 + 256 * warp) / kMxPadK + (lane >> 4);
        if ((lane & 15) == 0 && kt < nkt) *reinterpret_cast<uint32_t *>(scale_row + (size_t)kt * kMxTileBytes) = w;
    };
    if constexpr (kVals > 0) {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
            if (i * step < Kp) finish(i * step, v[i]);
    } else {
        for (int c0 = 0; c0 < Kp; c0 += step) {
            load_h(c0 + 8 * threadIdx.x, v[0]);
            finish(c0, v[0]);
        }
    }
    // Zero scale bytes for the rows past the last one: the CTAs of the last
    // 128-row block share them, a thread per word.
    const long long first = (long long)(a.rows - 1) / kMxTileRows * kMxTileRows;
    if (row >= first) {
        const int here = (int)(a.rows - first);
        uint8_t *tiles = a.scales + (size_t)(first / kMxTileRows) * nkt * kMxTileBytes;
        const int words = (kMxTileRows - here) * nkt;
        for (int i = (int)(row - first) * blockDim.x + threadIdx.x; i < words; i += here * blockDim.x) {
            const int p = here + i / nkt, kt = i % nkt;
            *reinterpret_cast<uint32_t *>(tiles + (size_t)kt * kMxTileBytes + 16 * (p & 31) + 4 * (p >> 5)) = 0u;
        }
    }
}

// Codes and scales back to values: a lane takes 8 values.
template <class T, bool kVec>
__global__ void __launch_bounds__(256)
    mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, T *__restrict__ y,
                         long long y_stride, int K, int bits, long long items) {
    const int Kp = mx_padded(K), nkt = Kp / kMxPadK, chunks = (Kp + 255) / 256;
    const long long item = blockIdx.x * 8LL + (threadIdx.x >> 5);
    pdl_wait();
    if (item >= items) return;
    const int c = (int)(item % chunks);
    const long long row = item / chunks;
    const int col = 256 * c + 8 * (threadIdx.x & 31);
    if (col >= Kp) return;
    const float s = mx_scale(scales[((size_t)(row / kMxTileRows) * nkt + col / kMxPadK) * kMxTileBytes +
                                    16 * (row & 31) + 4 * ((row & 127) >> 5) + ((col >> 5) & 3)]);
    float v[8];
    const uint8_t *p = codes + (size_t)row * Kp * bits / 8;
    if (bits == 4) {
        const uint32_t q = *reinterpret_cast<const uint32_t *>(p + (col >> 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = mx_from_e2m1x2((q >> (8 * i)) & 0xFFu);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(p + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = mx_from_e4m3x2(((i < 2 ? q.x : q.y) >> (16 * (i & 1))) & 0xFFFFu);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    store8<kVec>(y + row * y_stride, col, K, v);
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <class T>
bool rows_aligned(const void *p, long long stride) {
    return aligned16(p) && (stride * (long long)sizeof(T)) % 16 == 0;
}

// Grids are one-dimensional with 8 warps per CTA: at most 2^31 - 1 CTAs.
bool grid_of(long long items, unsigned *ctas) {
    const long long n = (items + 7) / 8;
    if (n > 0x7FFFFFFFLL) return false;
    *ctas = (unsigned)n;
    return true;
}

template <class T>
cudaError_t quantize_t(const LaunchCtx &c, const MxQuantizeArgs &a) {
    const int chunks = (mx_padded(a.K) + 255) / 256;
    const long long items = ((long long)a.rows + kMxTileRows - 1) / kMxTileRows * 32 * chunks;
    unsigned ctas;
    if (!grid_of(items, &ctas)) return cudaErrorInvalidValue;
    const bool vec = a.K % 8 == 0 && rows_aligned<T>(a.x, a.x_stride) && (!a.up || rows_aligned<T>(a.up, a.up_stride));
    auto kernel = a.up ? (vec ? mx_quantize_kernel<T, true, true> : mx_quantize_kernel<T, false, true>)
                       : (vec ? mx_quantize_kernel<T, true, false> : mx_quantize_kernel<T, false, false>);
    return launch_kernel(c, kernel, dim3(ctas), dim3(256), 0, static_cast<const T *>(a.x), a.x_stride,
                         static_cast<const T *>(a.up), a.up_stride, a.codes, a.scales, a.K, a.rows, a.bits, items);
}

template <class T>
cudaError_t rmsnorm_t(const LaunchCtx &c, const MxRmsnormArgs &a) {
    const bool vec = a.K % 8 == 0 && rows_aligned<T>(a.x, a.x_stride) &&
                     (!a.residual || (rows_aligned<T>(a.residual, a.residual_stride))) &&
                     (!a.h || rows_aligned<T>(a.h, a.h_stride)) && aligned16(a.weight);
    const RmsArgs k{a.x, a.residual, a.weight, a.h, a.x_stride, a.residual_stride, a.h_stride, a.codes, a.scales,
                    a.eps, a.K, a.rows, a.bits, a.weight_f32};
    const int Kp = mx_padded(a.K);
    // Threads: 8 values each up to 8192 wide, then more values per thread.
    int vals = 1;
    while (vals < 4 && Kp > 8 * 1024 * vals) vals *= 2;
    const bool kept = Kp <= 8 * 1024 * vals;
    int threads = kept ? (Kp / 8 + vals - 1) / vals : 1024;
    threads = (threads + 31) / 32 * 32;
    auto pick = [&](auto v1, auto v2, auto v4, auto v0) { return !kept ? v0 : vals == 1 ? v1 : vals == 2 ? v2 : v4; };
    auto kernel = vec ? pick(mx_rmsnorm_kernel<T, true, 1>, mx_rmsnorm_kernel<T, true, 2>,
                             mx_rmsnorm_kernel<T, true, 4>, mx_rmsnorm_kernel<T, true, 0>)
                      : pick(mx_rmsnorm_kernel<T, false, 1>, mx_rmsnorm_kernel<T, false, 2>,
                             mx_rmsnorm_kernel<T, false, 4>, mx_rmsnorm_kernel<T, false, 0>);
    return launch_kernel(c, kernel, dim3(a.rows), dim3(threads), 0, k);
}

template <class T>
cudaError_t dequantize_t(const LaunchCtx &c, const MxDequantizeArgs &a) {
    const long long items = (long long)a.rows * ((mx_padded(a.K) + 255) / 256);
    unsigned ctas;
    if (!grid_of(items, &ctas)) return cudaErrorInvalidValue;
    const bool vec = a.K % 8 == 0 && rows_aligned<T>(a.y, a.y_stride);
    return launch_kernel(c, vec ? mx_dequantize_kernel<T, true> : mx_dequantize_kernel<T, false>, dim3(ctas),
                         dim3(256), 0, a.codes, a.scales, static_cast<T *>(a.y), a.y_stride, a.K, a.bits, items);
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

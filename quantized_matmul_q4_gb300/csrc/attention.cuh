// What the attention kernels share: the batch's rows in tiles, powers of two
// as floats, codes to fp16.
//
// Numbers.  Codes times scales are exact in fp16 once a power of two is taken
// out: with `ref` the largest scale exponent of a group of tokens,
// k' = code · 2^(7 + e - ref) is at most 448 · 2^7 < 65504.  Where the tokens
// of a group differ by more than 2^kWide, each has a power of its own, so that
// no token, seen or not, costs another its bits; blocks 2^-17 below the
// largest of their token count as zero.  A query row is scaled by the power of two that puts its largest value into
// [2^14, 2^15): bf16 and fp16 rows are then exact to 2^-39 of that value, fp32
// rows are two fp16 numbers (22 bits).  The powers come back in the softmax, whose
// scores, maxima, sums and probabilities are fp32:
//
//   s = scale · log2 e · (q'·k') · 2^(powers of q and k)
//   u = s + vref                    vref: the power taken out of v
//   p = 2^(u - M + 6),  M >= max u - 8    (so p <= 2^14 in fp16)
//   O = Σ p v',  l = Σ p · 2^-vref,  y = O / l
//
// M is kept while no u passes it by more than 8, so O is rarely rescaled.
// A key whose v is far smaller than another's has a p that may be zero where its term
// of l is not.  So vref is kept within [kVrefLow, kVrefMax], 80 apart, which is what
// values from 2^-39 to 2^42 need (4 bits: 2^-45 to 2^36).  Rows that met others are taken
// once more, by plain_row.  Groups of zeros have kVrefMin, so that they raise M only where they are
// 2^60 and more times as probable as the rest.
// Probabilities enter the second product in fp16: one rounding to 2^-11 where y is 16 bits
// wide, two terms where it is fp32 (2^-22, of those above 2^-9 of the largest; the second
// term of smaller ones is below fp16's normal numbers).  A second term for 16-bit y as well would be
// half as much tensor work again.  Without it the error of an fp16 y is 2.55e-4 where that of fp32
// probabilities is 2.1e-4 (64 sequences of 4096), 2.8e-4 and 2.05e-4 over long keys of like probability;
// of a bf16 y half a percent larger.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "mx.cuh"
#include "mx_cache.cuh"
#include "sync.cuh"

namespace q4mm {

constexpr float kLog2e = 1.44269504f;
constexpr float kPShift = 6.f;      // log2 of p at u = M
constexpr float kPSlack = 8.f;      // u may pass M by this
constexpr int kVrefLow = -54;       // lowest power taken out of v
constexpr int kVrefMax = 26;        // highest
constexpr int kVrefMin = -80;       // that of zeros
constexpr int kWide = 4;            // a group's tokens share a power while their largest scales are within 2^this
constexpr int kNever = 0x7FFFFFFF;  // position of a NaN that there is not

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 2^e, e cut to a normal float's.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }

// x · 2^e, to below and above the normal floats.
__device__ __forceinline__ float scaled(float x, int e) { return x * pow2(e) * pow2(e - min(max(e, -126), 127)); }
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Value `at` of a 16-bit type.
__device__ __forceinline__ float wide_value(const void *p, MxType type, long long at) {
    return type == MxType::kF16 ? mx_float(static_cast<const __half *>(p)[at])
                                : mx_float(static_cast<const __nv_bfloat16 *>(p)[at]);
}

// Two E4M3 codes, or two E2M1 codes, as fp16.
__device__ __forceinline__ uint32_t half_e4m3x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t half_e4m3x2_high(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
template <int k>
__device__ __forceinline__ uint32_t half_e2m1x2(uint32_t bytes) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
        : "=r"(r)
        : "r"(bytes), "n"(k));
    return r;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two floats to fp16, the first in the low half.
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The largest scale byte of a word's first `blocks`, NaN bytes left out, and
// whether there is one of those.
struct ScaleWord {
    int b[4];
    int top;
    bool nan;
    __device__ __forceinline__ ScaleWord(uint32_t w, int blocks) {
        top = 0, nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = i < blocks ? (int)(w >> (8 * i) & 0xFF) : 0;
            nan |= b[i] == 255;
            top = max(top, b[i] == 255 ? 0 : b[i]);
        }
    }
};

// Whether values whose largest scale byte is `top` need another power.
__device__ __forceinline__ bool vref_passes(int top) {
    return top != 0 && (unsigned)(top - 134 - kVrefLow) > (unsigned)(kVrefMax - kVrefLow);
}

// A tile of `R` rows of one sequence and kv head.  Row r is token r / group of
// the sequence's new tokens, query head r % group of the kv head.
struct RowTile {
    int seq, first, rows;   // first row, rows (0: no such tile)
    int start, fresh, len;  // the sequence's first row of q, its new tokens, its cached tokens
};

// Tiles are numbered so that sequence i has those from starts[i]·group / R + i
// on: no fewer than its rows need, found by bisection instead of a prefix sum.
__device__ __forceinline__ RowTile row_tile(const MxBatchView &b, long long tile, int group, int R, int tokens) {
    RowTile t{};
    int i, s0, s1, len;
    long long from;
    if (b.seqs < 32) {  // starts and lengths by one load each, a lane each
        const int lane = threadIdx.x & 31;
        const int mine = lane <= b.seqs ? b.starts[lane] : 0, mine_len = lane < b.seqs ? b.lengths[lane] : 0;
        const long long mine_from = (long long)mine * group / R + lane;
        i = __popc(__ballot_sync(0xFFFFFFFFu, lane < b.seqs && mine_from <= tile)) - 1;
        if (i < 0) return t;
        s0 = __shfl_sync(0xFFFFFFFFu, mine, i), s1 = __shfl_sync(0xFFFFFFFFu, mine, i + 1);
        len = __shfl_sync(0xFFFFFFFFu, mine_len, i);
        from = (long long)s0 * group / R + i;
    } else {
        auto first_of = [&](int j) { return (long long)b.starts[j] * group / R + j; };
        i = warp_count_le(first_of, b.seqs, tile) - 1;
        if (i < 0) return t;
        s0 = b.starts[i], s1 = b.starts[i + 1], len = b.lengths[i], from = first_of(i);
    }
    if (s0 < 0 || s1 > tokens || s1 <= s0) return t;
    const long long first = (tile - from) * R, all = (long long)(s1 - s0) * group;
    if (first < 0 || first >= all) return t;
    t.seq = i, t.first = (int)first, t.rows = (int)min((long long)R, all - first);
    t.start = s0, t.fresh = s1 - s0, t.len = max(len, 0);
    return t;
}

// Keys that row r sees: positions below this (at most the table's).
__device__ __forceinline__ int keys_of(const RowTile &t, int r, int group, bool causal) {
    const int seen = causal ? t.len - t.fresh + r / group + 1 : t.len;
    return max(seen, 0);
}

// Sums of one row over some of its keys: y over those, four values a lane, and the M under which they count as 1.
struct PlainSums {
    float4 o;
    float m;
};

// By plain arithmetic, one row a warp: those of its first `keys` keys that lie in the groups of 16 tokens first, first +
// step .. before last.  Two passes, the second with probabilities that add up to 1, whose powers of two
// meet those of v before either leaves the floats.  Slow: decoding takes 17 times as long (16
// sequences of 2000, 32 heads: 53 and 896 us), a prompt of 2000 with 8 heads 412 times (33 us and 13.7 ms).
template <int kBits>
__device__ __forceinline__ PlainSums plain_row(const MxAttentionArgs &a, const RowTile &tile, const int row, const int group,
                                               const int head, const int keys, const int first, const int last,
                                               const int step) {
    const long long q_at = (long long)(tile.start + row / group) * a.q_token + (long long)(head * group + row % group) * a.q_head;
    const int sees = min(keys_of(tile, row, group, a.causal), keys);
    const int lane = threadIdx.x & 31, tok = lane & 15, half = lane >> 4;  // of K: a token, half the head
    const int D = a.cache.D, row_bytes = D * kBits / 8, per_page = a.cache.page / 16;
    constexpr int kWord = 32 / kBits;
    auto query = [&](int d) {
        return a.type == MxType::kF32 ? static_cast<const float *>(a.q)[q_at + d] : wide_value(a.q, a.type, q_at + d);
    };
    auto slot_of = [&](int g) -> long long {  // of the group's first token, or -1
        const int page = page_of(a.batch, a.cache, tile.seq, g / per_page, a.status);
        return page < 0 ? -1 : first_slot(a.cache, page, head) + 16 * (g % per_page);
    };
    auto score = [&](int g, long long slot) {
        if (slot < 0 || 16 * g + tok >= sees) slot = -1;
        float s = 0.f;
        if (slot >= 0) {
            const uint8_t *codes = a.cache.k_codes + (slot + tok) * row_bytes + half * (row_bytes / 2);
            const uint32_t scales = *reinterpret_cast<const uint32_t *>(a.cache.k_scales + (slot + tok) * 4);
            float block = 0.f;
            for (int i = 0; i < D / 2; i += kWord) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + i * kBits / 8);
                const int d = half * (D / 2) + i;
                float2 v[kWord / 2];
                if constexpr (kBits == 8)
                    v[0] = mx_from_e4m3x2<0>(w), v[1] = mx_from_e4m3x2<1>(w);
                else
                    v[0] = mx_from_e2m1x2<0>(w), v[1] = mx_from_e2m1x2<1>(w), v[2] = mx_from_e2m1x2<2>(w),
                    v[3] = mx_from_e2m1x2<3>(w);
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < kWord / 2; ++k) sum += v[k].x * query(d + 2 * k) + v[k].y * query(d + 2 * k + 1);
                block += sum;
                if ((d + kWord) % kMxBlock == 0 || i + kWord == D / 2)
                    s = fmaf(block, mx_scale(scales >> (8 * (d / kMxBlock)) & 0xFF), s), block = 0.f;
            }
        }
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
        return slot < 0 ? -INFINITY : s * (a.scale * kLog2e);  // (a scale of zero times an infinity is not one)
    };
    float m = -INFINITY, l = 0.f;
    for (int g = first; g < last && 16LL * g < sees; g += step) {
        const float s = score(g, slot_of(g));
        float top = s;
#pragma unroll
        for (int x = 1; x < 16; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        if (top > m) l *= m == -INFINITY ? 1.f : ex2(m - top), m = top;
        l += ex2(s - (m == -INFINITY ? 0.f : m));
    }
#pragma unroll
    for (int x = 1; x < 16; x *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    // What the keys' 2^score add up to, as a power of two: -infinity without keys, NaN where a score is.
    PlainSums r{make_float4(0.f, 0.f, 0.f, 0.f), l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + lg2(l)};
    for (int g = first; g < last && 16LL * g < sees; g += step) {
        const long long slot = slot_of(g);
        const float power = score(g, slot) - r.m;
        for (int j = 0; j < 16 && 16 * g + j < sees && slot >= 0; ++j) {
            const float t = __shfl_sync(0xFFFFFFFFu, power, j), whole = floorf(t);
            if (4 * lane >= D) continue;
            const uint8_t *codes = a.cache.v_codes + (slot + j) * row_bytes + lane * kBits / 2;
            float2 lo, hi;
            if constexpr (kBits == 8) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(codes);
                lo = mx_from_e4m3x2<0>(w), hi = mx_from_e4m3x2<1>(w);
            } else {
                const uint32_t w = *reinterpret_cast<const uint16_t *>(codes);
                lo = mx_from_e2m1x2<0>(w), hi = mx_from_e2m1x2<1>(w);
            }
            const int b = a.cache.v_scales[(slot + j) * 4 + 4 * lane / kMxBlock], e = (int)fmaxf(whole, -999.f) + b - 127;
            const float p = b == 255 ? __int_as_float(0x7FC00000) : ex2(t - whole);
            r.o.x += scaled(lo.x * p, e), r.o.y += scaled(lo.y * p, e);
            r.o.z += scaled(hi.x * p, e), r.o.w += scaled(hi.y * p, e);
        }
    }
    return r;
}

// Four neighbouring outputs.
__device__ __forceinline__ void store4(void *y, MxType type, long long at, bool vec, float4 v) {
    if (type == MxType::kF32) {
        float *p = static_cast<float *>(y) + at;
        if (vec)
            *reinterpret_cast<float4 *>(p) = v;
        else
            p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
        return;
    }
    uint32_t lo, hi;
    if (type == MxType::kF16)
        lo = mx_pack2<__half>(v.x, v.y), hi = mx_pack2<__half>(v.z, v.w);
    else
        lo = mx_pack2<__nv_bfloat16>(v.x, v.y), hi = mx_pack2<__nv_bfloat16>(v.z, v.w);
    uint16_t *p = static_cast<uint16_t *>(y) + at;
    if (vec)
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    else
        p[0] = (uint16_t)lo, p[1] = (uint16_t)(lo >> 16), p[2] = (uint16_t)hi, p[3] = (uint16_t)(hi >> 16);
}

}  // namespace q4mm

// Rotary positions, and the paged MX cache written and read (sm_103a).
//
//   rope_rotate     pairs (u, v) of a head at position p, frequency f:
//                   u' = m (u cos pf - v sin pf), v' = m (v cos pf + u sin pf)
//   mx_cache_write  k turned so, k and v quantised in blocks of 32 along the
//                   head, to their slots of the cache's pages
//   mx_cache_read   the values back
//
// All move each byte once and are meant to be bound by HBM.  A lane holds
// eight consecutive values of a head (16 bytes of a 16-bit type), a power of
// two of lanes a head, so the two halves of a rotated head meet in one warp
// and a block of 32 is four lanes.  A CTA takes a few consecutive tokens of
// all heads: their angles are computed once, and in the cache the tokens of a
// head lie next to each other.
//
// Rope of 8192 x 32 x 128 bf16: 22.5 us in a chain of calls (88% of the measured copy rate),
// 25.7 a call (77%); 20748 tokens of 8 heads read from 8 bits to bf16: 24.1 (78%); 8272
// tokens of 32 heads rotated and written from fp16 to 8 bits: 46.4 (65%), 64% of the issue
// slots and the loads' latency (each lane holds 32 to 64 bytes of loads, 32 warps an SM).
//
// Angles.  p·f in radians needs some 20 bits before the point for far
// positions and 24 behind it.  So f / 2π, in turns, is taken as a 64-bit
// fraction, and the product with the integer p modulo 2^64 is the angle
// modulo a turn, exactly: what is left is the rounding of f / 2π to a multiple
// of 2^-64 (times p).  The fraction's nearest quarter turn goes off as an
// integer; the rest, at most π/4, goes through the Taylor series of sine and
// cosine (their next terms, x^11 / 11! and x^12 / 12!, are below 2^-29), so c
// and s are within 2·2^-24.
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "mx_cache.cuh"

namespace q4mm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 16;   // tokens a CTA takes together
constexpr int kMaxPairs = 128;   // rotated pairs of a head

// f / 2π modulo 1 in units of 2^-64 turns, for the bits of a double f: its
// 53-bit significand times 2^66 / 2π = 2^64 · 0.6366..., in integers (the
// chip's fp64 rate is two per clock and SM).  Subnormal f count as 0.
__device__ __forceinline__ uint64_t turns_of(double f) {
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const int e = (int)(bits >> 52 & 0x7FF) - 1023;
    if (e < -1022) return 0;
    const uint64_t m = bits << 11 | 1ull << 63;                       // f = m · 2^(e - 63)
    const uint64_t hi = __umul64hi(m, 0xA2F9836E4E441529ull);        // 2^66 / 2π
    const int up = e - 1;
    const uint64_t t = up >= 0 ? (up < 64 ? hi << up : 0) : (up > -64 ? hi >> -up : 0);
    return bits >> 63 ? 0 - t : t;
}

// cos and sin of `turn` · 2^-64 turns, times m.
__device__ __forceinline__ float2 cos_sin(uint64_t turn, float m) {
    const int32_t a = (int32_t)(turn >> 32);
    const int32_t q = (a >> 29) + 1 >> 1;                                        // nearest quarter
    // The rest in radians as x + xl, both roundings on the way kept.
    const int32_t r = (int32_t)((uint32_t)a - ((uint32_t)q << 30));
    constexpr float kRad = 1.46291807926715968e-9f;                        // 2π / 2^32,
    constexpr float kRadRest = (float)(1.46291807926715968105e-9 - (double)kRad);  // and what it lacks
    const float hi = (float)r, lo = (float)(r - (int32_t)hi);
    const float x = hi * kRad, xl = fmaf(hi, kRad, -x) + fmaf(hi, kRadRest, lo * kRad);
    const float z = x * x;
    float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
    s = fmaf(s, z, 8.33333333e-3f), s = fmaf(s, z, -1.66666667e-1f);
    s = x + fmaf(x * z, s, xl);                                            // (xl's factor, cos x, is 0.7 at least)
    float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
    c = fmaf(c, z, -1.38888889e-3f), c = fmaf(c, z, 4.16666667e-2f), c = fmaf(c, z, -0.5f);
    c = 1.f + fmaf(c, z, -x * xl);
    float co = q & 1 ? s : c, si = q & 1 ? c : s;     // a quarter on: (c, s) -> (-s, c)
    if ((q & 3) == 1 || (q & 3) == 2) co = -co;
    if (q & 2) si = -si;
    return make_float2(co * m, si * m);
}

// Angles of the tokens of a CTA.
struct Angles {
    float cos[kMaxTokens][kMaxPairs], sin[kMaxTokens][kMaxPairs];
};

// Fills the table for `tokens` tokens at position(s).
template <class F>
__device__ __forceinline__ void fill_angles(Angles &t, const RopeView &r, int tokens, F position) {
    const int pairs = r.rotated / 2;
    for (int e = threadIdx.x; e < tokens * pairs; e += kThreads) {
        const int s = e / pairs, i = e - s * pairs;
        const double f = r.frequencies[i];
        float2 cs = cos_sin((uint64_t)position(s) * turns_of(f), r.magnitude);
        if (!isfinite(f)) cs = make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
        t.cos[s][i] = cs.x, t.sin[s][i] = cs.y;
    }
}

// Eight values of a head as they lie in memory.
template <class T>
struct Eight {
    uint4 w[sizeof(T) / 2];
};

template <class T>
__device__ __forceinline__ Eight<T> fetch8(const T *p) {
    Eight<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = ld_stream_u4(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
// As above from any address, `n` values at stride 1, zeros behind them.
template <class T>
__device__ __forceinline__ Eight<T> fetch8_each(const T *p, int n) {
    Eight<T> r;
    T *v = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : mx_from_float<T>(0.f);
    return r;
}
template <class T>
__device__ __forceinline__ void floats8(const Eight<T> &r, float (&v)[8]) {
    const T *p = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mx_float(p[i]);
}

template <bool kVec, class T>
__device__ __forceinline__ void put8(T *p, int n, const float (&v)[8]) {
    if constexpr (kVec) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(p) = make_uint4(mx_pack2<T>(v[0], v[1]), mx_pack2<T>(v[2], v[3]),
                                                       mx_pack2<T>(v[4], v[5]), mx_pack2<T>(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = mx_from_float<T>(v[i]);
    }
}

// A lane's eight values d .. d + 7 of a head, and what the rotation of split
// halves needs beside them: the values half a rotated part away.
template <bool kVec, class T>
struct Turned8 {
    Eight<T> own, other;

    __device__ __forceinline__ void load(const T *head, int d, int D, const RopeView &r) {
        const int half = r.rotated / 2;
        if constexpr (kVec) {
            own = fetch8(head + d);
            if (!r.interleaved && d < r.rotated) other = fetch8(head + (d < half ? d + half : d - half));
        } else {
            own = fetch8_each(head + d, D - d);
            if (!r.interleaved && d < r.rotated) {
                T *v = reinterpret_cast<T *>(&other);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = d + i;
                    v[i] = e < r.rotated ? head[e < half ? e + half : e - half] : mx_from_float<T>(0.f);
                }
            }
        }
    }

    // The turned values, with the angles of one token.
    __device__ __forceinline__ void turn(const float *cos, const float *sin, int d, const RopeView &r,
                                         float (&v)[8]) const {
        floats8(own, v);
        if (d >= r.rotated) return;
        const int half = r.rotated / 2;
        if (r.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                if (d + i < r.rotated) {
                    const float c = cos[(d + i) / 2], s = sin[(d + i) / 2], a = v[i], b = v[i + 1];
                    v[i] = fmaf(a, c, -(b * s)), v[i + 1] = fmaf(b, c, a * s);
                }
            }
        } else {
            float o[8];
            floats8(other, o);
            if constexpr (kVec) {  // all eight on one side
                const float sign = d < half ? -1.f : 1.f;
                const int i0 = d < half ? d : d - half;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 c = *reinterpret_cast<const float4 *>(cos + i0 + i);
                    const float4 s = *reinterpret_cast<const float4 *>(sin + i0 + i);
                    v[i] = fmaf(v[i], c.x, sign * (o[i] * s.x));
                    v[i + 1] = fmaf(v[i + 1], c.y, sign * (o[i + 1] * s.y));
                    v[i + 2] = fmaf(v[i + 2], c.z, sign * (o[i + 2] * s.z));
                    v[i + 3] = fmaf(v[i + 3], c.w, sign * (o[i + 3] * s.w));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = d + i;
                    if (e < r.rotated) {
                        const float c = cos[e < half ? e : e - half], s = sin[e < half ? e : e - half];
                        v[i] = fmaf(v[i], c, e < half ? -(o[i] * s) : o[i] * s);
                    }
                }
            }
        }
    }
};

// How the lanes of a CTA's warps share the heads of its tokens (a power of
// two): each lane stays with one token and takes every step-th vector, so
// that its addresses advance by constants.
struct Items {
    int d;          // the lane's first value
    int token;      // of the CTA's
    int first, step;
    __device__ __forceinline__ Items(int lanes_log, int tokens_log) {
        const int lane = threadIdx.x & 31, subs = 32 >> lanes_log;
        const int q = (blockIdx.y * kWarps + threadIdx.x / 32) * subs + (lane >> lanes_log);
        d = 8 * (lane & ((1 << lanes_log) - 1));
        token = q & ((1 << tokens_log) - 1), first = q >> tokens_log;
        step = (gridDim.y * kWarps * subs) >> tokens_log;
    }
};

// A lane's values d .. d + 7 of a head and, half a head on, its partners in
// the rotation of split halves: both are turned by the same angles.
template <class T>
struct TurnedPairs {
    Eight<T> u, v;
    __device__ __forceinline__ void load(const T *head, int d, int half) {
        u = fetch8(head + d), v = fetch8(head + d + half);
    }
    __device__ __forceinline__ void turn(const float *cos, const float *sin, int d, float (&a)[8], float (&b)[8]) const {
        float x[8], y[8];
        floats8(u, x), floats8(v, y);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(cos + d + i);
            const float4 s = *reinterpret_cast<const float4 *>(sin + d + i);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float2 c2 = j ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
                const float2 s2 = j ? make_float2(s.z, s.w) : make_float2(s.x, s.y);
                const float2 x2 = make_float2(x[i + j], x[i + j + 1]), y2 = make_float2(y[i + j], y[i + j + 1]);
                const float2 ys = __fmul2_rn(y2, s2), xs = __fmul2_rn(x2, s2);
                const float2 p = ffma2(x2, c2, make_float2(-ys.x, -ys.y)), q = ffma2(y2, c2, xs);
                a[i + j] = p.x, a[i + j + 1] = p.y, b[i + j] = q.x, b[i + j + 1] = q.y;
            }
        }
    }
};

// kForm: 2 for split halves of whole heads, a lane with both partners (lanes
// for half a head); 1 for aligned heads; 0 for any.
template <class T, int kForm>
__global__ void __launch_bounds__(kThreads) rope_rotate_kernel(const RopeArgs a, const int lanes_log,
                                                               const int tokens_log) {
    constexpr int kU = 2;
    __shared__ __align__(16) Angles table;
    pdl_wait();
    const long long t0 = (long long)blockIdx.x << tokens_log;
    const int tokens = (int)min((long long)1 << tokens_log, a.tokens - t0);
    fill_angles(table, a.rope, tokens, [&](int s) {
        return a.positions_64 ? static_cast<const long long *>(a.positions)[t0 + s]
                              : (long long)static_cast<const int *>(a.positions)[t0 + s];
    });
    __syncthreads();
    const Items it(lanes_log, tokens_log);
    const int s = it.token, span = kForm == 2 ? a.D / 2 : a.D;
    const bool mine = s < tokens && it.d < span;
    const T *x = static_cast<const T *>(a.x) + (t0 + s) * a.x_token + it.first * a.x_head;
    T *out = static_cast<T *>(a.out) + (t0 + s) * a.out_token + it.first * a.out_head;
    // (Out may be x: a head is read whole, by lanes of one warp, before any of it is written.)
    for (int h = it.first; __any_sync(0xFFFFFFFFu, h < a.heads); h += kU * it.step) {
        bool ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) ok[u] = mine && h + u * it.step < a.heads;
        if constexpr (kForm == 2) {
            TurnedPairs<T> v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (ok[u]) v[u].load(x + u * it.step * a.x_head, it.d, span);
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (!ok[u]) continue;
                float f[8], g[8];
                v[u].turn(table.cos[s], table.sin[s], it.d, f, g);
                put8<true>(out + u * it.step * a.out_head + it.d, 8, f);
                put8<true>(out + u * it.step * a.out_head + it.d + span, 8, g);
            }
        } else {
            Turned8<kForm == 1, T> v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (ok[u]) v[u].load(x + u * it.step * a.x_head, it.d, a.D, a.rope);
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (!ok[u]) continue;
                float f[8];
                v[u].turn(table.cos[s], table.sin[s], it.d, a.rope, f);
                put8<kForm == 1>(out + u * it.step * a.out_head + it.d, a.D - it.d, f);
            }
        }
        x += kU * it.step * a.x_head, out += kU * it.step * a.out_head;
    }
}

// Where the tokens of a CTA lie: their positions, and slots of head 0 (below 0: nowhere).
struct Places {
    long long slot[kMaxTokens];
    int position[kMaxTokens];
};

__device__ __forceinline__ void find_places(Places &p, const MxBatchView &b, const MxCacheView &c, long long t0,
                                            int tokens, int *status) {
    for (int s = threadIdx.x / 32; s < tokens; s += kWarps) {
        int i, len = 0, end = 0;
        if (b.seqs < 32) {  // starts and lengths by one load each, a lane each
            const int lane = threadIdx.x & 31;
            const int start = lane <= b.seqs ? b.starts[lane] : 0x7FFFFFFF, mine = lane < b.seqs ? b.lengths[lane] : 0;
            i = __popc(__ballot_sync(0xFFFFFFFFu, start <= t0 + s && lane <= b.seqs)) - 1;
            len = __shfl_sync(0xFFFFFFFFu, mine, max(i, 0)), end = __shfl_sync(0xFFFFFFFFu, start, (i + 1) & 31);
            if (i >= b.seqs) i = -1;
        } else {
            i = sequence_of_row(b, t0 + s);
            if (i >= 0) len = b.lengths[i], end = b.starts[i + 1];
        }
        long long slot = -1;
        int pos = 0;
        if (i >= 0) {
            pos = (int)max((long long)len - end + (t0 + s), -1LL);
            if (pos >= 0) {
                const int page = page_of(b, c, i, pos / c.page, status);
                if (page >= 0) slot = first_slot(c, page, 0) + pos % c.page;
            }
        }
        if ((threadIdx.x & 31) == 0) p.slot[s] = slot, p.position[s] = pos;
    }
    __syncthreads();
}

// As cos_sin of a magnitude of 1, in 64 bits to some 2^-27: the last additions
// with what they round off, the square and the rest's factor in full.
__device__ __forceinline__ double2 cos_sin_more(uint64_t turn) {
    const int32_t a = (int32_t)(turn >> 32), q = (a >> 29) + 1 >> 1, r = (int32_t)((uint32_t)a - ((uint32_t)q << 30));
    constexpr float kRad = 1.46291807926715968e-9f;
    constexpr float kRadRest = (float)(1.46291807926715968105e-9 - (double)kRad);
    const float hi = (float)r, lo = (float)(r - (int32_t)hi) + (float)(uint32_t)turn * 0x1p-32f;
    const float x = hi * kRad, xl = fmaf(hi, kRad, -x) + fmaf(hi, kRadRest, lo * kRad);
    const float z = x * x, zl = fmaf(x, x, -z);
    float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
    s = fmaf(s, z, 8.33333333e-3f), s = fmaf(s, z, -1.66666667e-1f);
    const float sl = fmaf(x * z, s, xl * fmaf(z, -0.5f, 1.f));
    float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
    c = fmaf(c, z, -1.38888889e-3f), c = fmaf(c, z, 4.16666667e-2f);
    const float cl = fmaf(c * z, z, fmaf(zl, -0.5f, -x * xl));
    const double co = (1.0 - 0.5 * (double)z) + (double)cl, si = (double)x + (double)sl;
    const double u = q & 1 ? si : co, v = q & 1 ? co : si;
    return make_double2((q & 3) == 1 || (q & 3) == 2 ? -u : u, q & 2 ? -v : v);
}

// Value d of a head, turned, rounded to odd: a code made of it is that of the
// value before.  Out of line, for the few that need it.
template <class T>
__device__ __noinline__ float turned_again(const T *head, int d, const RopeView r, long long position) {
    const int half = r.rotated / 2, i = r.interleaved ? d / 2 : d < half ? d : d - half;
    const bool first = r.interleaved ? d % 2 == 0 : d < half;
    const int other = r.interleaved ? d ^ 1 : first ? d + half : d - half;
    const double2 cs = cos_sin_more((uint64_t)position * turns_of(r.frequencies[i]));
    const double a = mx_float(head[d]), b = mx_float(head[other]);
    const double v = r.magnitude * (first ? a * cs.x - b * cs.y : a * cs.x + b * cs.y);
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Turned values that lie within 4 units of a border between two codes, where
// the fp32 arithmetic may fall on its other side, are taken again: nine in
// 2^20 (8 bits) or 2^22.  (Without this 26 to 40 codes of 68 million differed from
// those of the exact values, with it 9 to 19; 8272 tokens written take 46.4 us, 43.2 without.)
// Below the codes' normal numbers the borders lie elsewhere and are left as they are.
// So are those within 4 units of a power of two where that is the block's largest value: there
// the block's scale has its border, and all of its codes with it.  Returns the float bits of
// the block's largest value.
template <int kBits, class T>
__device__ __forceinline__ uint32_t settle(float (&f)[8], const T *head, int d, const RopeView &r, long long position, bool ok) {
    constexpr uint32_t kMask = kBits == 8 ? 0xFFFFF : 0x3FFFFF, kBorder = kMask / 2 + 1;
    const uint32_t amax = mx_block_amax(f);
    uint32_t nearest = kMask;
#pragma unroll
    for (int i = 0; i < 8; ++i) nearest = min(nearest, __float_as_uint(f[i]) - (kBorder - 4) & kMask);
    const bool top = (amax + 4 & 0x7FFFFF) <= 8 && amax >= 0x00800000u;
    // (Values that are not turned lie on borders often: a 16-bit one in 16.)
    if (!__any_sync(0xFFFFFFFFu, (nearest <= 8 || top) && d < r.rotated)) return amax;
    const bool mine = ok && (position != 0 || r.magnitude != 1.f);  // (else they are as they were)
    const uint32_t power = top ? amax + 4 & 0x7F800000u : 0x80000000u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (mine && d + i < r.rotated && ((__float_as_uint(f[i]) - (kBorder - 4) & kMask) <= 8 ||
                                          (__float_as_uint(f[i]) & 0x7FFFFFFFu) + 4 - power <= 8))
            f[i] = turned_again(head, d + i, r, position);
    return mx_block_amax(f);
}

// Quantises eight values of a block of four lanes, whose largest has the bits amax, into a slot: codes at
// `codes`, the block's scale byte (and the padding's zeros) at `scales`.
template <int kBits>
__device__ __forceinline__ void put_codes(const float (&f)[8], uint32_t amax, uint8_t *codes, uint8_t *scales, int d, int D,
                                          bool ok) {
    const uint32_t b = mx_quantize8(f, amax, kBits, codes, d, ok ? D : 0);
    if (ok && (d & 31) == 0) {
        const int block = d / kMxBlock, blocks = D / kMxBlock;
        scales[block] = (uint8_t)b;
        for (int pad = block + blocks; pad < 4; pad += blocks) scales[pad] = 0;
    }
}

// kForm as for rope_rotate, for the keys.
template <class T, int kForm, int kBits>
__global__ void __launch_bounds__(kThreads, kForm == 0 ? 1 : 4) mx_cache_write_kernel(const MxCacheIoArgs a, const RopeView rope,
                                                                  const int lanes_log, const int tokens_log) {
    __shared__ __align__(16) Angles table;
    __shared__ Places at;
    pdl_wait();
    const long long t0 = (long long)blockIdx.x << tokens_log;
    const int tokens = (int)min((long long)1 << tokens_log, a.tokens - t0);
    find_places(at, a.batch, a.cache, t0, tokens, a.status);
    if (rope.rotated) {
        fill_angles(table, rope, tokens, [&](int s) { return (long long)at.position[s]; });
        __syncthreads();
    }
    const int D = a.cache.D, H = a.cache.heads, row_bytes = D * kBits / 8;
    auto heads = [&](const Items &it, const void *from, long long token, long long head, uint8_t *codes, uint8_t *scales,
                     auto pairs, const RopeView &r) {
        constexpr bool kPairs = decltype(pairs)::value;
        constexpr int kU = kPairs ? 2 : 4;
        const int s = it.token, span = kPairs ? D / 2 : D;
        const bool mine = s < tokens && it.d < span && at.slot[s < tokens ? s : 0] >= 0;
        const T *x = static_cast<const T *>(from) + (t0 + s) * token + it.first * head;
        const long long slot = mine ? at.slot[s] + (long long)it.first * a.cache.page : 0;
        const long long apart = (long long)it.step * a.cache.page;  // slots between the lane's heads
        codes += slot * row_bytes, scales += slot * 4;
        for (int h = it.first; __any_sync(0xFFFFFFFFu, h < H); h += kU * it.step) {
            bool ok[kU];
            std::conditional_t<kPairs, TurnedPairs<T>, Turned8<kForm != 0, T>> v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                ok[u] = mine && h + u * it.step < H;
                if (!ok[u]) continue;
                if constexpr (kPairs)
                    v[u].load(x + u * it.step * head, it.d, span);
                else
                    v[u].load(x + u * it.step * head, it.d, D, r);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = 0.f;
                uint8_t *c = codes + u * apart * row_bytes, *b = scales + u * apart * 4;
                if constexpr (kPairs) {
                    float g[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = 0.f;
                    if (ok[u]) v[u].turn(table.cos[s], table.sin[s], it.d, f, g);
                    const uint32_t f_max = settle<kBits>(f, x + u * it.step * head, it.d, r, at.position[s], ok[u]);
                    put_codes<kBits>(f, f_max, c, b, it.d, D, ok[u]);
                    const uint32_t g_max = settle<kBits>(g, x + u * it.step * head, it.d + span, r, at.position[s], ok[u]);
                    put_codes<kBits>(g, g_max, c, b, it.d + span, D, ok[u]);
                } else {
                    if (ok[u]) v[u].turn(table.cos[s], table.sin[s], it.d, r, f);
                    const uint32_t f_max = r.rotated ? settle<kBits>(f, x + u * it.step * head, it.d, r, at.position[s], ok[u])
                                                     : mx_block_amax(f);
                    put_codes<kBits>(f, f_max, c, b, it.d, D, ok[u]);
                }
            }
            x += kU * it.step * head, codes += kU * apart * row_bytes, scales += kU * apart * 4;
        }
    };
    const RopeView still{nullptr, 0, false, 1.f};
    if constexpr (kForm == 2)
        heads(Items(lanes_log - 1, tokens_log), a.k, a.k_token, a.k_head, a.cache.k_codes, a.cache.k_scales,
              std::true_type{}, rope);
    else
        heads(Items(lanes_log, tokens_log), a.k, a.k_token, a.k_head, a.cache.k_codes, a.cache.k_scales,
              std::false_type{}, rope);
    heads(Items(lanes_log, tokens_log), a.v, a.v_token, a.v_head, a.cache.v_codes, a.cache.v_scales, std::false_type{},
          still);
}

template <class T, bool kVec, int kBits>
__global__ void __launch_bounds__(kThreads) mx_cache_read_kernel(const MxCacheIoArgs a, const int lanes_log,
                                                                 const int tokens_log) {
    constexpr int kU = 4;
    __shared__ Places at;
    pdl_wait();
    const long long t0 = (long long)blockIdx.x << tokens_log;
    const int tokens = (int)min((long long)1 << tokens_log, a.tokens - t0);
    find_places(at, a.batch, a.cache, t0, tokens, a.status);
    const Items it(lanes_log, tokens_log);
    const int D = a.cache.D, H = a.cache.heads, s = it.token, row_bytes = D * kBits / 8;
    if (s >= tokens || it.d >= D || at.slot[s] < 0) return;
    const long long slot = at.slot[s] + (long long)it.first * a.cache.page, apart = (long long)it.step * a.cache.page;
    auto heads = [&](const uint8_t *codes, const uint8_t *scales, const void *to, long long token, long long head) {
        codes += slot * row_bytes + it.d * kBits / 8, scales += slot * 4 + it.d / kMxBlock;
        T *y = static_cast<T *>(const_cast<void *>(to)) + (t0 + s) * token + it.first * head + it.d;
        for (int h = it.first; h < H; h += kU * it.step) {
            uint2 q[kU];
            uint32_t b[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (h + u * it.step >= H) continue;
                const uint8_t *p = codes + u * apart * row_bytes;
                if constexpr (kBits == 8)
                    q[u] = __ldg(reinterpret_cast<const uint2 *>(p));
                else
                    q[u].x = __ldg(reinterpret_cast<const uint32_t *>(p));
                b[u] = __ldg(scales + u * apart * 4);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (h + u * it.step >= H) continue;
                float2 g[4];
                if constexpr (kBits == 4) {
                    g[0] = mx_from_e2m1x2<0>(q[u].x), g[1] = mx_from_e2m1x2<1>(q[u].x);
                    g[2] = mx_from_e2m1x2<2>(q[u].x), g[3] = mx_from_e2m1x2<3>(q[u].x);
                } else {
                    g[0] = mx_from_e4m3x2<0>(q[u].x), g[1] = mx_from_e4m3x2<1>(q[u].x);
                    g[2] = mx_from_e4m3x2<0>(q[u].y), g[3] = mx_from_e4m3x2<1>(q[u].y);
                }
                const float scale = mx_scale(b[u]);
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 z = __fmul2_rn(g[i], make_float2(scale, scale));
                    f[2 * i] = z.x, f[2 * i + 1] = z.y;
                }
                put8<kVec>(y + u * it.step * head, D - it.d, f);
            }
            codes += kU * apart * row_bytes, scales += kU * apart * 4, y += kU * it.step * head;
        }
    };
    heads(a.cache.k_codes, a.cache.k_scales, a.k, a.k_token, a.k_head);
    heads(a.cache.v_codes, a.cache.v_scales, a.v, a.v_token, a.v_head);
}

// Every head of every token starts on 16 bytes.
bool heads_aligned(const void *p, long long token, long long head, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token * (long long)size % 16 == 0 &&
           head * (long long)size % 16 == 0;
}

// Tokens a CTA takes (the most, up to 8, that leave two CTAs an SM, else 1; up to 16
// where 8 tokens' heads are less than a pass of its lanes: 28934 tokens of 2 heads
// written 27.9 us, 35.2 with 8, read 12.0 and 16.7) and
// CTAs that share them (up to two an SM, each with work for its warps).  2048
// tokens written, 32 heads of 128: 18.7 us with 1 token a CTA, 13.5 with 2, 12.9 with 4, 16.6
// with 8 (256 CTAs); 8272 (without settle): 67.4, 44.5, 43.1, 43.6; 20748 read, 8 heads:
// 78, 52, 33, 24.7; rope of 1000 tokens: 4.6, 3.8, 4.8, 6.9.
struct Shape {
    int lanes_log, tokens_log;
    dim3 grid;
};
Shape shape_of(const LaunchCtx &c, int tokens, int vectors, int D, int unroll) {
    Shape s{};
    while (8 << s.lanes_log < D) ++s.lanes_log;
    const int lanes = kWarps * (32 >> s.lanes_log);  // vectors of a pass, apart from `unroll`
    s.tokens_log = 16 <= lanes && vectors * 8 < lanes * unroll ? 4 : 3;
    while (s.tokens_log > 0 && ((long long)tokens + (1 << s.tokens_log) - 1) >> s.tokens_log < 2 * c.num_sms) --s.tokens_log;
    const int x = (tokens + (1 << s.tokens_log) - 1) >> s.tokens_log;
    const long long per_cta = (long long)kWarps * (32 >> s.lanes_log) * unroll;  // items of one pass
    const long long most = (((long long)vectors << s.tokens_log) + per_cta - 1) / per_cta;
    long long y = (2LL * c.num_sms + x - 1) / x;
    y = y < most ? y : most;
    s.grid = dim3((unsigned)x, (unsigned)(y < 65535 ? y : 65535));
    return s;
}

// Split halves of whole aligned heads of 8 · 2^n values each.
bool whole_halves(const RopeView &r, int D) { return !r.interleaved && r.rotated == D && D >= 16 && (D & (D - 1)) == 0; }

template <class T>
cudaError_t rope_t(const LaunchCtx &c, const RopeArgs &a) {
    const bool vec = a.D % 8 == 0 && heads_aligned(a.x, a.x_token, a.x_head, sizeof(T)) &&
                     heads_aligned(a.out, a.out_token, a.out_head, sizeof(T)) &&
                     (a.rope.interleaved || a.rope.rotated % 16 == 0);
    const bool pairs = vec && whole_halves(a.rope, a.D);
    const Shape s = shape_of(c, a.tokens, a.heads, pairs ? a.D / 2 : a.D, 2);
    auto kernel = pairs ? rope_rotate_kernel<T, 2> : vec ? rope_rotate_kernel<T, 1> : rope_rotate_kernel<T, 0>;
    return launch_kernel(c, kernel, s.grid, dim3(kThreads), 0, a, s.lanes_log, s.tokens_log);
}

template <class T>
cudaError_t write_t(const LaunchCtx &c, const MxCacheIoArgs &a, const RopeView &rope) {
    const bool vec = heads_aligned(a.k, a.k_token, a.k_head, sizeof(T)) &&
                     heads_aligned(a.v, a.v_token, a.v_head, sizeof(T)) &&
                     (rope.interleaved || rope.rotated % 16 == 0);
    // (A block is four lanes, so half a head is one block at least.)
    const bool pairs = vec && whole_halves(rope, a.cache.D) && a.cache.D >= 64;
    const Shape s = shape_of(c, a.tokens, a.cache.heads, a.cache.D, 2);
    auto pick = [&](auto f2, auto f1, auto f0) { return pairs ? f2 : vec ? f1 : f0; };
    auto kernel = a.cache.bits == 4
                      ? pick(mx_cache_write_kernel<T, 2, 4>, mx_cache_write_kernel<T, 1, 4>, mx_cache_write_kernel<T, 0, 4>)
                      : pick(mx_cache_write_kernel<T, 2, 8>, mx_cache_write_kernel<T, 1, 8>, mx_cache_write_kernel<T, 0, 8>);
    return launch_kernel(c, kernel, s.grid, dim3(kThreads), 0, a, rope, s.lanes_log, s.tokens_log);
}

template <class T>
cudaError_t read_t(const LaunchCtx &c, const MxCacheIoArgs &a) {
    const bool vec = heads_aligned(a.k, a.k_token, a.k_head, sizeof(T)) &&
                     heads_aligned(a.v, a.v_token, a.v_head, sizeof(T));
    const Shape s = shape_of(c, a.tokens, a.cache.heads, a.cache.D, 4);
    auto kernel = a.cache.bits == 4 ? (vec ? mx_cache_read_kernel<T, true, 4> : mx_cache_read_kernel<T, false, 4>)
                                    : (vec ? mx_cache_read_kernel<T, true, 8> : mx_cache_read_kernel<T, false, 8>);
    return launch_kernel(c, kernel, s.grid, dim3(kThreads), 0, a, s.lanes_log, s.tokens_log);
}

}  // namespace

cudaError_t launch_rope_rotate(const LaunchCtx &c, MxType type, const RopeArgs &a) {
    return type == MxType::kF32   ? rope_t<float>(c, a)
           : type == MxType::kF16 ? rope_t<__half>(c, a)
                                  : rope_t<__nv_bfloat16>(c, a);
}

cudaError_t launch_mx_cache_write(const LaunchCtx &c, MxType type, const MxCacheIoArgs &a, const RopeView &rope) {
    return type == MxType::kF32   ? write_t<float>(c, a, rope)
           : type == MxType::kF16 ? write_t<__half>(c, a, rope)
                                  : write_t<__nv_bfloat16>(c, a, rope);
}

cudaError_t launch_mx_cache_read(const LaunchCtx &c, MxType type, const MxCacheIoArgs &a) {
    return type == MxType::kF32   ? read_t<float>(c, a)
           : type == MxType::kF16 ? read_t<__half>(c, a)
                                  : read_t<__nv_bfloat16>(c, a);
}

}  // namespace q4mm

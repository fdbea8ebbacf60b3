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
// Angles.  p·f in radians needs some 20 bits before the point for far
// positions and 24 behind it.  So f / 2π, in turns, is taken as a 64-bit
// fraction, and the product with the integer p modulo 2^64 is the angle
// modulo a turn, exactly: what is left is the rounding of f / 2π to a multiple
// of 2^-64 (times p).  The fraction's nearest quarter turn goes off as an
// integer; the rest, at most π/4, goes through the Taylor series of sine and
// cosine (their next terms, x^11 / 11! and x^12 / 12!, are below 2^-29), so c
// and s are within 2·2^-24.
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "mx_cache.cuh"

namespace q4mm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 8;    // tokens a CTA takes together
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
    const float x = (float)(int32_t)((uint32_t)a - ((uint32_t)q << 30)) * 1.46291807926715968e-9f;  // 2π / 2^32
    const float z = x * x;
    float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
    s = fmaf(s, z, 8.33333333e-3f), s = fmaf(s, z, -1.66666667e-1f);
    s = fmaf(x * z, s, x);
    float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
    c = fmaf(c, z, -1.38888889e-3f), c = fmaf(c, z, 4.16666667e-2f), c = fmaf(c, z, -0.5f);
    c = fmaf(c, z, 1.f);
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

// How a warp's lanes share the heads of a CTA's tokens: item r is token
// r % tokens (a power of two) of vector r / tokens, lanes of 8 values each.
struct Items {
    int sub, subs, d;  // which of the warp's items this lane serves, how many it has, the lane's first value
    __device__ __forceinline__ explicit Items(int lanes_log) {
        const int lane = threadIdx.x & 31;
        sub = lane >> lanes_log, subs = 32 >> lanes_log, d = 8 * (lane & ((1 << lanes_log) - 1));
    }
};

template <class T, bool kVec>
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
    const Items it(lanes_log);
    const long long rows = (long long)a.heads << tokens_log;
    const T *x = static_cast<const T *>(a.x);
    T *out = static_cast<T *>(a.out);
    const long long each = (long long)gridDim.y * kWarps * it.subs * kU;
    for (long long r0 = ((long long)blockIdx.y * kWarps + threadIdx.x / 32) * it.subs * kU; r0 < rows; r0 += each) {
        Turned8<kVec, T> v[kU];
        bool ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const long long r = r0 + u * it.subs + it.sub, h = r >> tokens_log;
            const int s = (int)(r & ((1 << tokens_log) - 1));
            ok[u] = r < rows && s < tokens && it.d < a.D;
            if (ok[u]) v[u].load(x + (t0 + s) * a.x_token + h * a.x_head, it.d, a.D, a.rope);
        }
        __syncwarp();  // out may be x: a head is read whole before any of it is written
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (!ok[u]) continue;
            const long long r = r0 + u * it.subs + it.sub, h = r >> tokens_log;
            const int s = (int)(r & ((1 << tokens_log) - 1));
            float f[8];
            v[u].turn(table.cos[s], table.sin[s], it.d, a.rope, f);
            put8<kVec>(out + (t0 + s) * a.out_token + h * a.out_head + it.d, a.D - it.d, f);
        }
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
        const int i = sequence_of_row(b, t0 + s);
        long long slot = -1;
        int pos = 0;
        if (i >= 0) {
            pos = (int)max((long long)b.lengths[i] - b.starts[i + 1] + (t0 + s), -1LL);
            if (pos >= 0) {
                const int page = page_of(b, c, i, pos / c.page, status);
                if (page >= 0) slot = first_slot(c, page, 0) + pos % c.page;
            }
        }
        if ((threadIdx.x & 31) == 0) p.slot[s] = slot, p.position[s] = pos;
    }
    __syncthreads();
}

template <class T, bool kVec, int kBits>
__global__ void __launch_bounds__(kThreads) mx_cache_write_kernel(const MxCacheIoArgs a, const RopeView rope,
                                                                  const int lanes_log, const int tokens_log) {
    constexpr int kU = 2;
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
    const Items it(lanes_log);
    const int D = a.cache.D, blocks = D / kMxBlock, H = a.cache.heads;
    const long long rows = (long long)2 * H << tokens_log;
    const long long each = (long long)gridDim.y * kWarps * it.subs * kU;
    const RopeView still{nullptr, 0, false, 1.f};
    for (long long r0 = ((long long)blockIdx.y * kWarps + threadIdx.x / 32) * it.subs * kU; r0 < rows; r0 += each) {
        Turned8<kVec, T> v[kU];
        bool ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const long long r = r0 + u * it.subs + it.sub;
            const int s = (int)(r & ((1 << tokens_log) - 1)), hv = (int)(r >> tokens_log);
            const bool is_v = hv >= H;
            const int h = is_v ? hv - H : hv;
            ok[u] = r < rows && s < tokens && it.d < D && at.slot[s < tokens ? s : 0] >= 0;
            if (ok[u]) {
                const T *head = static_cast<const T *>(is_v ? a.v : a.k) + (t0 + s) * (is_v ? a.v_token : a.k_token) +
                                h * (is_v ? a.v_head : a.k_head);
                v[u].load(head, it.d, D, is_v ? still : rope);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const long long r = r0 + u * it.subs + it.sub;
            const int s = (int)(r & ((1 << tokens_log) - 1)), hv = (int)(r >> tokens_log);
            const bool is_v = hv >= H;
            const int h = is_v ? hv - H : hv;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
            if (ok[u]) v[u].turn(table.cos[s], table.sin[s], it.d, is_v ? still : rope, f);
            const uint32_t amax = mx_block_amax(f);
            const long long slot = ok[u] ? at.slot[s] + (long long)h * a.cache.page : 0;
            uint8_t *codes = (is_v ? a.cache.v_codes : a.cache.k_codes) + slot * (D * kBits / 8);
            const uint32_t b = mx_quantize8(f, amax, kBits, codes, it.d, ok[u] ? D : 0);
            if (ok[u] && (it.d & 31) == 0) {
                uint8_t *scales = (is_v ? a.cache.v_scales : a.cache.k_scales) + slot * 4;
                const int block = it.d / kMxBlock;
                scales[block] = (uint8_t)b;
                for (int pad = block + blocks; pad < 4; pad += blocks) scales[pad] = 0;
            }
        }
    }
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
    const Items it(lanes_log);
    const int D = a.cache.D, H = a.cache.heads;
    const long long rows = (long long)2 * H << tokens_log;
    const long long each = (long long)gridDim.y * kWarps * it.subs * kU;
    for (long long r0 = ((long long)blockIdx.y * kWarps + threadIdx.x / 32) * it.subs * kU; r0 < rows; r0 += each) {
        uint2 q[kU];
        uint32_t b[kU];
        bool ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const long long r = r0 + u * it.subs + it.sub;
            const int s = (int)(r & ((1 << tokens_log) - 1)), hv = (int)(r >> tokens_log);
            const bool is_v = hv >= H;
            ok[u] = r < rows && s < tokens && it.d < D && at.slot[s < tokens ? s : 0] >= 0;
            q[u] = make_uint2(0u, 0u), b[u] = 0;
            if (ok[u]) {
                const long long slot = at.slot[s] + (long long)(is_v ? hv - H : hv) * a.cache.page;
                const uint8_t *p = (is_v ? a.cache.v_codes : a.cache.k_codes) + (slot * D + it.d) * kBits / 8;
                if constexpr (kBits == 8)
                    q[u] = __ldg(reinterpret_cast<const uint2 *>(p));
                else
                    q[u].x = __ldg(reinterpret_cast<const uint32_t *>(p));
                b[u] = __ldg((is_v ? a.cache.v_scales : a.cache.k_scales) + slot * 4 + it.d / kMxBlock);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (!ok[u]) continue;
            const long long r = r0 + u * it.subs + it.sub;
            const int s = (int)(r & ((1 << tokens_log) - 1)), hv = (int)(r >> tokens_log);
            const bool is_v = hv >= H;
            const int h = is_v ? hv - H : hv;
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
            for (int i = 0; i < 4; ++i) f[2 * i] = g[i].x * scale, f[2 * i + 1] = g[i].y * scale;
            T *head = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k)) +
                      (t0 + s) * (is_v ? a.v_token : a.k_token) + h * (is_v ? a.v_head : a.k_head);
            put8<kVec>(head + it.d, D - it.d, f);
        }
    }
}

// Every head of every token starts on 16 bytes.
bool heads_aligned(const void *p, long long token, long long head, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token * (long long)size % 16 == 0 &&
           head * (long long)size % 16 == 0;
}

// Tokens a CTA takes (8 where that leaves two CTAs an SM, else 1) and CTAs
// that share them (up to two an SM, each with work for its warps).
struct Shape {
    int lanes_log, tokens_log;
    dim3 grid;
};
Shape shape_of(const LaunchCtx &c, int tokens, int vectors, int D, int unroll) {
    Shape s{};
    while (8 << s.lanes_log < D) ++s.lanes_log;
    s.tokens_log = (tokens + 7) / 8 >= 2 * c.num_sms ? 3 : 0;
    const int x = (tokens + (1 << s.tokens_log) - 1) >> s.tokens_log;
    const long long per_cta = (long long)kWarps * (32 >> s.lanes_log) * unroll;  // items of one pass
    const long long most = (((long long)vectors << s.tokens_log) + per_cta - 1) / per_cta;
    long long y = (2LL * c.num_sms + x - 1) / x;
    y = y < most ? y : most;
    s.grid = dim3((unsigned)x, (unsigned)(y < 65535 ? y : 65535));
    return s;
}

template <class T>
cudaError_t rope_t(const LaunchCtx &c, const RopeArgs &a) {
    const bool vec = a.D % 8 == 0 && heads_aligned(a.x, a.x_token, a.x_head, sizeof(T)) &&
                     heads_aligned(a.out, a.out_token, a.out_head, sizeof(T)) &&
                     (a.rope.interleaved || a.rope.rotated % 16 == 0);
    const Shape s = shape_of(c, a.tokens, a.heads, a.D, 2);
    auto kernel = vec ? rope_rotate_kernel<T, true> : rope_rotate_kernel<T, false>;
    return launch_kernel(c, kernel, s.grid, dim3(kThreads), 0, a, s.lanes_log, s.tokens_log);
}

template <class T>
cudaError_t write_t(const LaunchCtx &c, const MxCacheIoArgs &a, const RopeView &rope) {
    const bool vec = heads_aligned(a.k, a.k_token, a.k_head, sizeof(T)) &&
                     heads_aligned(a.v, a.v_token, a.v_head, sizeof(T)) &&
                     (rope.interleaved || rope.rotated % 16 == 0);
    const Shape s = shape_of(c, a.tokens, 2 * a.cache.heads, a.cache.D, 2);
    auto kernel = a.cache.bits == 4 ? (vec ? mx_cache_write_kernel<T, true, 4> : mx_cache_write_kernel<T, false, 4>)
                                    : (vec ? mx_cache_write_kernel<T, true, 8> : mx_cache_write_kernel<T, false, 8>);
    return launch_kernel(c, kernel, s.grid, dim3(kThreads), 0, a, rope, s.lanes_log, s.tokens_log);
}

template <class T>
cudaError_t read_t(const LaunchCtx &c, const MxCacheIoArgs &a) {
    const bool vec = heads_aligned(a.k, a.k_token, a.k_head, sizeof(T)) &&
                     heads_aligned(a.v, a.v_token, a.v_head, sizeof(T));
    const Shape s = shape_of(c, a.tokens, 2 * a.cache.heads, a.cache.D, 4);
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

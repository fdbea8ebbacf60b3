// Attention over a paged MX cache for few rows a key/value head (sm_103a):
// decoding, 8 or 16 rows a tile.
//
// Every byte of the cache is read once by the tile that needs it, so the
// kernel is meant to be bound by HBM: 8-bit heads of 128 bring an SM some 23
// values per clock, of which each costs 1.3 instructions here.  Codes go from
// global memory straight into the fragments of mma.sync (m16n8k16, fp16 in,
// fp32 out); a tensor instruction with its operands in shared memory would
// have to pad 8 rows to 128.  With the tokens or head values on M and the rows
// on N:
//
//   Sᵀ[token][row] = K Qᵀ      16 tokens x 8 rows, 16 values of the head a step
//   Oᵀ[value][row] = Vᵀ Pᵀ     16 values x 8 rows, 16 tokens a step
//
// The order of head values within a step, and of values among the M rows, is
// free as long as both operands agree, so a lane takes runs that it can load
// whole: of K, 32 neighbouring values of two tokens (lane group g holds tokens
// g and g + 8), of V, 16 neighbouring values of four tokens, whose codes two
// tokens at a time are interleaved by a byte permute and converted together.
// Pᵀ's fragment is Sᵀ's transposed in 8 x 8 pieces by movmatrix.
//
// Warps take groups of 16 tokens in turn, the next group's codes on their way
// while one is computed; each keeps a maximum, sum and accumulator of its own.
// They are joined in shared memory, and the CTAs of a cluster, which share a
// tile's keys, through distributed shared memory, in a fixed order.
#include <cstdint>

#include "attention.cuh"
#include "attention_geometry.h"
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "sync.cuh"

namespace q4mm {

namespace {

constexpr int kThreads = 32 * kFewWarps;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// kWords words from p (kWords·4 bytes aligned, 16 at most).
template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t *p, bool ok, uint32_t (&w)[kWords]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
    if (!ok) return;
    if constexpr (kWords >= 4) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 v = ld_stream_u4(p + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    } else if constexpr (kWords == 2) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
        w[0] = ld_stream_u32(p);
    }
}

__device__ __forceinline__ float value_at(const void *p, MxType type, long long i) {
    return type == MxType::kF32   ? static_cast<const float *>(p)[i]
           : type == MxType::kF16 ? __half2float(static_cast<const __half *>(p)[i])
                                  : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_at(void *p, MxType type, long long i, float v) {
    if (type == MxType::kF32)
        static_cast<float *>(p)[i] = v;
    else if (type == MxType::kF16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// kDP: the head's values rounded up to 64 or 128; kNR: row tiles of 8; kNP:
// fp16 terms of a query value and a probability.
template <int kDP, int kNR, int kNP>
struct FewShared {
    static constexpr int kR = 8 * kNR;
    static constexpr int kPitch = kDP + 8;  // halves of a staged query row
    union {
        __half q[kNP][kR][kPitch];
        float o[kFewWarps][kR][kDP];  // each warp's sums; the CTA's in [0]
    };
    float m[kFewWarps][kR], l[kFewWarps][kR];
    float m_all[kR], l_all[kR];
    int power[kR];   // of two, taken out of a query row
    int nan_from[4]; // first position whose v has NaN in a block
};

template <int kBits, int kDP, int kNR, int kNP>
__global__ void __launch_bounds__(kThreads, kNR == 1 && kNP == 1 ? 2 : 1)
    mx_attention_few_kernel(const MxAttentionArgs a, const int group) {
    using Shared = FewShared<kDP, kNR, kNP>;
    constexpr int kR = Shared::kR;
    constexpr int kSteps = kDP / 16;             // of 16 head values
    constexpr int kKRun = kDP / 4, kVRun = kDP / 8;  // neighbouring values of a lane
    constexpr int kKW = kKRun * kBits / 32, kVW = kVRun * kBits / 32;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int D = a.cache.D, blocks = D / kMxBlock;

    pdl_wait();
    const long long item = blockIdx.x / S;
    const int head = (int)(item % a.cache.heads);
    const RowTile tile = row_tile(a.batch, item / a.cache.heads, group, kR, a.tokens);
    if (tile.rows == 0) return;  // with the whole cluster

    // Query rows to fp16, each by a power of two of its own.
    for (int r = warp; r < kR; r += kFewWarps) {
        constexpr int kEach = kDP / 32;
        float v[kEach];
        uint32_t top = 0;
        const int row = tile.first + r;
        const long long at = (long long)(tile.start + row / group) * a.q_token +
                             (long long)(head * group + row % group) * a.q_head;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int d = lane + 32 * i;
            v[i] = r < tile.rows && d < D ? value_at(a.q, a.type, at + d) : 0.f;
            top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        // 2^(141 - e) puts a largest value of biased exponent e at 2^14; not where it is infinite or NaN.
        const int e = top >= 0x7F800000u ? 141 : max((int)(top >> 23), 15);
        const float mult = __int_as_float((268 - e) << 23);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const float x = v[i] * mult;
            const __half hi = __float2half_rn(x);
            sh.q[0][r][lane + 32 * i] = hi;
            if constexpr (kNP == 2) sh.q[1][r][lane + 32 * i] = __float2half_rn(x - __half2float(hi));
        }
        if (lane == 0) sh.power[r] = e - 141;
    }
    if (threadIdx.x < 4) sh.nan_from[threadIdx.x] = kNever;
    __syncthreads();

    uint32_t qf[kNP][kNR][kSteps][2];
    int power[kNR][2], sees[kNR][2];  // of this lane's rows 2t and 2t + 1
    int keys = 0;                     // that any row sees
#pragma unroll
    for (int n = 0; n < kNR; ++n) {
#pragma unroll
        for (int p = 0; p < kNP; ++p)
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const uint2 w = *reinterpret_cast<const uint2 *>(&sh.q[p][8 * n + g][t * kKRun + 4 * k]);
                qf[p][n][k][0] = w.x, qf[p][n][k][1] = w.y;
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * n + 2 * t + j;
            power[n][j] = sh.power[r];
            sees[n][j] = r < tile.rows ? keys_of(tile, tile.first + r, group, a.causal) : 0;
        }
    }
    keys = keys_of(tile, tile.first + tile.rows - 1, group, a.causal);
    const long long room = (long long)a.batch.width * a.cache.page;
    if (keys > room) {
        if (threadIdx.x == 0) atomicOr(a.status, kStatusIndex);
        keys = (int)room;
    }
    __syncthreads();  // the staged rows have been read: their memory is the sums'

    const int groups = (keys + kFewGroup - 1) / kFewGroup;
    const int g0 = (int)((long long)groups * rank / S), g1 = (int)((long long)groups * (rank + 1) / S);
    const float c0 = a.scale * kLog2e;

    float o[kNR][kSteps][4];
    float M[kNR][2], l[kNR][2];
#pragma unroll
    for (int n = 0; n < kNR; ++n) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
        M[n][0] = M[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
    }

    // The warp's groups: codes of one on their way while another is used.
    uint32_t kw[2][kKW], vw[4][kVW], sw = 0;
    const int per_page = a.cache.page / kFewGroup, row_bytes = D * kBits / 8;
    int piece = (g0 + warp) / per_page, within = (g0 + warp) % per_page;  // page and group within it
    const bool k_in = t * kKRun < D, v_in = g * kVRun < D;
    auto next_page = [&](int gi) { return gi < g1 ? page_of(a.batch, a.cache, tile.seq, piece, a.status) : -1; };
    auto advance = [&]() {
        within += kFewWarps % per_page, piece += kFewWarps / per_page;
        if (within >= per_page) within -= per_page, ++piece;
    };
    int gi = g0 + warp;
    int page = next_page(gi);
    long long slot = first_slot(a.cache, page, head) + kFewGroup * within;
    auto load_k = [&](int left) {  // tokens of the group that exist
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_words<kKW>(a.cache.k_codes + (slot + g + 8 * i) * row_bytes + t * kKRun * kBits / 8,
                            k_in && g + 8 * i < left, kw[i]);
    };
    auto load_v = [&](int left) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
            load_words<kVW>(a.cache.v_codes + (slot + tok) * row_bytes + g * kVRun * kBits / 8, v_in && tok < left,
                            vw[i]);
        }
    };
    // Scales: lane i < 16 has token i's word for k, lane 16 + i for v.
    auto load_s = [&](int left) {
        sw = 0;
        if ((lane & 15) < left)
            sw = ld_stream_u32((lane < 16 ? a.cache.k_scales : a.cache.v_scales) + (slot + (lane & 15)) * 4);
    };
    auto tokens_left = [&](int gi_, int page_) { return page_ < 0 || gi_ >= g1 ? 0 : keys - kFewGroup * gi_; };
    int left = tokens_left(gi, page);
    load_k(left), load_s(left), load_v(left);

    for (; gi < g1; gi += kFewWarps) {
        const int here = left, base = kFewGroup * gi;
        // This group's scales: of each token the power taken out, and four
        // bytes of exponents 33 above those of its blocks' multipliers.
        const ScaleWord s(sw, blocks);
        const bool is_v = lane >= 16;
        int ref = s.top - 134;
        if (is_v) ref = max(ref, kVrefMin);
        uint32_t mults = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int e = max(s.b[i] - 127 - ref + 33, 0);
            if (s.b[i] == 255) e = is_v ? 0 : 161;  // infinite: times a zero code NaN
            mults |= (uint32_t)e << (8 * i);
        }
        if (__any_sync(0xFFFFFFFFu, is_v && s.nan)) {  // NaN in v reaches the rows that see it, and no others
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (is_v && s.b[i] == 255) atomicMin(&sh.nan_from[i], base + (lane & 15));
        }
        auto mult_of = [&](int from, int block) {  // a multiplier in both halves
            const uint32_t w = __shfl_sync(0xFFFFFFFFu, mults, from);
            const float f = __int_as_float(((w >> (8 * block) & 0xFF) + 94) << 23);
            return half2_of(f, f);
        };
        int kref[2], vref[2];
        uint32_t km[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kref[i] = __shfl_sync(0xFFFFFFFFu, ref, g + 8 * i), vref[i] = __shfl_sync(0xFFFFFFFFu, ref, 16 + g + 8 * i);
            km[i] = mult_of(g + 8 * i, t * kKRun / kMxBlock);
        }
        uint32_t vm[2];  // of tokens 2t and 2t + 1, and of those 8 on
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = mult_of(16 + 2 * t + 8 * i, g * kVRun / kMxBlock);
            const uint32_t hi = mult_of(17 + 2 * t + 8 * i, g * kVRun / kMxBlock);
            vm[i] = __byte_perm(lo, hi, 0x5410);
        }

        float sc[kNR][4];
#pragma unroll
        for (int n = 0; n < kNR; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            uint32_t f[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (kBits == 8) {
                    f[i][0] = half_e4m3x2(kw[i][k]), f[i][1] = half_e4m3x2_high(kw[i][k]);
                } else if (k % 2 == 0) {
                    f[i][0] = half_e2m1x2<0>(kw[i][k / 2]), f[i][1] = half_e2m1x2<1>(kw[i][k / 2]);
                } else {
                    f[i][0] = half_e2m1x2<2>(kw[i][k / 2]), f[i][1] = half_e2m1x2<3>(kw[i][k / 2]);
                }
                f[i][0] = half2_mul(f[i][0], km[i]), f[i][1] = half2_mul(f[i][1], km[i]);
            }
#pragma unroll
            for (int n = 0; n < kNR; ++n)
#pragma unroll
                for (int p = 0; p < kNP; ++p)
                    mma_16816(sc[n], f[0][0], f[1][0], f[0][1], f[1][1], qf[p][n][k][0], qf[p][n][k][1]);
        }

        // The next group: its page, then K and the scales; V once this one's is used.
        advance();
        page = next_page(gi + kFewWarps);
        slot = first_slot(a.cache, page, head) + kFewGroup * within;
        left = tokens_left(gi + kFewWarps, page);
        load_k(left), load_s(left);

        float u[kNR][4];
        bool more = false;
#pragma unroll
        for (int n = 0; n < kNR; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = j >> 1, tok = g + 8 * i;
                const float s2 = sc[n][j] * c0 * pow2(power[n][j & 1] + kref[i]) + (float)vref[i];
                u[n][j] = tok < here && base + tok < sees[n][j & 1] ? s2 : -INFINITY;
                more |= u[n][j] > M[n][j & 1] + kPSlack;
            }
        if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
            for (int n = 0; n < kNR; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = fmaxf(u[n][j], u[n][2 + j]);
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                    m = fmaxf(m, M[n][j]);
                    const float by = M[n][j] == -INFINITY ? 0.f : ex2(M[n][j] - m);
                    M[n][j] = m, l[n][j] *= by;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) o[n][i][j] *= by, o[n][i][2 + j] *= by;
                }
        }
        uint32_t pf[kNP][kNR][2];
#pragma unroll
        for (int n = 0; n < kNR; ++n) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float m = M[n][j & 1];
                p[j] = ex2(u[n][j] - ((m == -INFINITY ? 0.f : m) - kPShift));
                l[n][j & 1] = fmaf(p[j], pow2(-vref[j >> 1]), l[n][j & 1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t hi = half2_of(p[2 * i], p[2 * i + 1]);
                pf[0][n][i] = transposed(hi);
                if constexpr (kNP == 2) {
                    const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    pf[1][n][i] = transposed(half2_of(p[2 * i] - back.x, p[2 * i + 1] - back.y));
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            uint32_t f[2][2];  // tokens' pair, value 2k or 2k + 1 of the lane's
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (kBits == 8) {
                    const uint32_t w = __byte_perm(vw[2 * i][k / 2], vw[2 * i + 1][k / 2], k % 2 ? 0x7362 : 0x5140);
                    f[i][0] = half_e4m3x2(w), f[i][1] = half_e4m3x2_high(w);
                } else {
                    const uint32_t x = vw[2 * i][k / 4], y = vw[2 * i + 1][k / 4];
                    const uint32_t even = (x & 0x0F0F0F0Fu) | (y & 0x0F0F0F0Fu) << 4;
                    const uint32_t odd = (x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
                    f[i][0] = k % 4 == 0 ? half_e2m1x2<0>(even) : k % 4 == 1 ? half_e2m1x2<1>(even)
                              : k % 4 == 2 ? half_e2m1x2<2>(even) : half_e2m1x2<3>(even);
                    f[i][1] = k % 4 == 0 ? half_e2m1x2<0>(odd) : k % 4 == 1 ? half_e2m1x2<1>(odd)
                              : k % 4 == 2 ? half_e2m1x2<2>(odd) : half_e2m1x2<3>(odd);
                }
                f[i][0] = half2_mul(f[i][0], vm[i]), f[i][1] = half2_mul(f[i][1], vm[i]);
            }
#pragma unroll
            for (int n = 0; n < kNR; ++n)
#pragma unroll
                for (int p = 0; p < kNP; ++p)
                    mma_16816(o[n][k], f[0][0], f[0][1], f[1][0], f[1][1], pf[p][n][0], pf[p][n][1]);
        }
        load_v(left);
    }

    // Sums over a warp's tokens, then over the warps, then over the cluster.
#pragma unroll
    for (int n = 0; n < kNR; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v = l[n][j];
#pragma unroll
            for (int x = 4; x < 32; x *= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, x);
            const int r = 8 * n + 2 * t + j;
            if (g == 0) sh.m[warp][r] = M[n][j], sh.l[warp][r] = v;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                *reinterpret_cast<float2 *>(&sh.o[warp][r][g * kVRun + 2 * i]) = make_float2(o[n][i][j], o[n][i][2 + j]);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < tile.rows * (kDP / 4); i += kThreads) {
        const int r = i / (kDP / 4), d = 4 * (i % (kDP / 4));
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, sh.m[w][r]);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float ls = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float by = sh.m[w][r] == -INFINITY ? 0.f : ex2(sh.m[w][r] - m);
            const float4 v = *reinterpret_cast<const float4 *>(&sh.o[w][r][d]);
            // (A warp without a maximum has zeros, or NaN where its scores are.)
            ls += sh.m[w][r] == -INFINITY ? sh.l[w][r] : by * sh.l[w][r];
            sum.x = fmaf(by, v.x, sum.x), sum.y = fmaf(by, v.y, sum.y);
            sum.z = fmaf(by, v.z, sum.z), sum.w = fmaf(by, v.w, sum.w);
        }
        *reinterpret_cast<float4 *>(&sh.o[0][r][d]) = sum;
        if (d == 0) sh.m_all[r] = m, sh.l_all[r] = ls;
    }
    if (S > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const uint32_t o_at = smem_addr(sh.o), m_at = smem_addr(sh.m_all), l_at = smem_addr(sh.l_all),
                   n_at = smem_addr(sh.nan_from);
    for (int i = rank * kThreads + threadIdx.x; i < tile.rows * (kDP / 4); i += S * kThreads) {
        const int r = i / (kDP / 4), d = 4 * (i % (kDP / 4));
        if (d >= D) continue;
        float m = -INFINITY;
        int nan_from = kNever;
        for (int s = 0; s < S; ++s) {
            m = fmaxf(m, ld_cluster_f32(map_to_rank(m_at + 4 * r, s)));
            nan_from = min(nan_from, __float_as_int(ld_cluster_f32(map_to_rank(n_at + 4 * (d / kMxBlock), s))));
        }
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float ls = 0.f;
        for (int s = 0; s < S; ++s) {
            const float mi = ld_cluster_f32(map_to_rank(m_at + 4 * r, s)), li = ld_cluster_f32(map_to_rank(l_at + 4 * r, s));
            const float4 v = ld_cluster_v4(map_to_rank(o_at + 4 * (r * kDP + d), s));
            const float by = mi == -INFINITY ? 0.f : ex2(mi - m);
            ls += mi == -INFINITY ? li : by * li;
            sum.x = fmaf(by, v.x, sum.x), sum.y = fmaf(by, v.y, sum.y);
            sum.z = fmaf(by, v.z, sum.z), sum.w = fmaf(by, v.w, sum.w);
        }
        const int row = tile.first + r;
        if (nan_from < keys_of(tile, row, group, a.causal)) ls = __int_as_float(0x7FC00000);
        const long long at = (long long)(tile.start + row / group) * a.y_token +
                             (long long)(head * group + row % group) * a.y_head + d;
        // A row that sees nothing has no sum: zeros.
        const float by = ls == 0.f ? 0.f : 1.f / ls;
        store_at(a.y, a.type, at, sum.x * by), store_at(a.y, a.type, at + 1, sum.y * by);
        store_at(a.y, a.type, at + 2, sum.z * by), store_at(a.y, a.type, at + 3, sum.w * by);
    }
    if (S > 1) cluster_sync_all();  // no CTA leaves while another reads its sums
}

template <int kBits, int kDP, int kNR, int kNP>
cudaError_t launch_few(const LaunchCtx &c, const MxAttentionArgs &a) {
    auto kernel = mx_attention_few_kernel<kBits, kDP, kNR, kNP>;
    constexpr size_t bytes = sizeof(FewShared<kDP, kNR, kNP>);
    cudaError_t e = ensure_smem(kernel, bytes);
    if (e != cudaSuccess) return e;
    const int group = a.heads / a.cache.heads;
    const long long tiles = (long long)a.tokens * group / (8 * kNR) + a.batch.seqs;
    // (A table's width bounds the keys; their number is the device's to know.)
    const long long keys = (long long)a.batch.width * a.cache.page;
    const int S = few_split(tiles, a.cache.heads, (int)(keys < 0x7FFFFFFF ? keys : 0x7FFFFFFF), c.num_sms);
    const long long ctas = tiles * a.cache.heads * S;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (S > 8 && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, group);
}

template <int kBits, int kDP>
cudaError_t launch_rows(const LaunchCtx &c, const MxAttentionArgs &a) {
    const long long rows = (long long)a.tokens * (a.heads / a.cache.heads);
    const bool wide = rows > 8LL * a.batch.seqs;  // more than 8 rows a sequence and kv head
    if (a.type == MxType::kF32)
        return wide ? launch_few<kBits, kDP, 2, 2>(c, a) : launch_few<kBits, kDP, 1, 2>(c, a);
    return wide ? launch_few<kBits, kDP, 2, 1>(c, a) : launch_few<kBits, kDP, 1, 1>(c, a);
}

}  // namespace

cudaError_t launch_mx_attention_few(const LaunchCtx &c, const MxAttentionArgs &a) {
    const bool narrow = a.cache.D <= 64;
    if (a.cache.bits == 4) return narrow ? launch_rows<4, 64>(c, a) : launch_rows<4, 128>(c, a);
    return narrow ? launch_rows<8, 64>(c, a) : launch_rows<8, 128>(c, a);
}

}  // namespace q4mm
